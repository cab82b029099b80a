"""The serving calls on the GPU against their plain 64-bit forms: page plans
and appends exactly, attention within the bounds of its arithmetic
(serve_harness.attend_bounds), and all of them together with the index build
and decode."""
import math

import numpy as np
import pytest
import torch

import retrieval_sparse_attention_wave_b200 as W
from tests import serve_harness as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------- page plans

def make_table(have, page, n_pages, max_pages, seed):
    """A table whose requests hold pages for `have` tokens, and the other pages
    on the stack in a shuffled order (with stale entries behind its end)."""
    rng = np.random.default_rng(seed)
    order = rng.permutation(n_pages).astype(np.int32)
    bt = np.full((len(have), max_pages), -1, dtype=np.int32)
    at = 0
    for b, h in enumerate(have):
        n = -(-h // page)
        bt[b, :n] = order[at:at + n]
        at += n
    free = order[at:]
    stack = np.concatenate([free, order[:2]])
    return W.PageTable(i32(bt), i32(have), i32(stack), i32([len(free)]), page, n_pages)


def check_plan(table, new, capacity, **kw):
    bt = table.block_table.tolist()
    ref = S.plan_reference(bt, table.seq_lens.tolist(), new, table.free_pages.tolist(),
                           int(table.n_free), table.page_size, table.n_pages, capacity)
    p = W.plan_pages(table, i32(new), capacity, **kw)
    got = [x.tolist() for x in (table.block_table, p.slot_map, p.positions, p.starts, p.seq_lens)]
    for name, a, b in zip(("table", "slots", "positions", "starts", "lens"), got, ref):
        assert a == b, name
    assert int(p.n_free) == ref[5]
    return p


@pytest.mark.parametrize("page", [1, 4, 16, 1024])
@pytest.mark.parametrize("have,new", [
    ([0], [1]), ([0], [0]), ([15], [1]), ([16], [1]), ([17, 0, 31, 5], [1, 40, 1, 0]),
    ([0, 0, 0], [0, 700, 0]), ([1000, 3], [5000, 2999]),
])
def test_plan(page, have, new):
    need = sum(-(-(h + n) // page) for h, n in zip(have, new))
    table = make_table(have, page, need + 4, max(-(-(h + n) // page) for h, n in zip(have, new)) + 1, 1)
    ws = W.serve_workspace(DEV)
    for pad in (0, 3):
        check_plan(table, new, sum(new) + pad, ws=ws)
        table.block_table.copy_(make_table(have, page, need + 4, table.block_table.shape[1], 1).block_table)
    assert W.read_device_status(ws) == 0


def test_plan_full_batch_advances_in_place():
    rng = np.random.default_rng(3)
    have = rng.integers(0, 200, 256).tolist()
    table = make_table(have, 16, 9000, 60, 4)
    ws = W.serve_workspace(DEV)
    for step in range(4):
        new = (rng.integers(0, 2, 256) * (rng.integers(1, 120, 256) if step == 1 else 1)).tolist()
        before = table.seq_lens.tolist()
        check_plan(table, new, sum(new) + 700, update=True, ws=ws)
        assert table.seq_lens.tolist() == [h + n for h, n in zip(before, new)]
    assert W.read_device_status(ws) == 0


def test_plan_captured_step_advances_with_each_replay():
    table = make_table([30, 0, 17], 16, 40, 8, 5)
    new = i32([1, 1, 0])
    plan = W.PagePlan.empty(table, 4, update=True)
    ws = W.serve_workspace(DEV)
    ref_table = table.block_table.tolist()
    lens, stack, n_free = table.seq_lens.tolist(), table.free_pages.tolist(), int(table.n_free)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        W.plan_pages(table, new, 4, out=plan, update=True, ws=ws)
    assert table.seq_lens.tolist() == lens
    for _ in range(20):
        ref_table, slots, positions, _, lens, n_free = S.plan_reference(
            ref_table, lens, [1, 1, 0], stack, n_free, 16, 40, 4)
        g.replay()
        assert plan.slot_map.tolist() == slots and plan.positions.tolist() == positions
        assert table.seq_lens.tolist() == lens and int(table.n_free) == n_free
    assert table.block_table.tolist() == ref_table
    assert W.read_device_status(ws) == 0


@pytest.mark.parametrize("what,flag", [
    ("pages", W.WI_DEV_NO_PAGES), ("capacity", W.WI_DEV_NO_PAGES), ("row", W.WI_DEV_NO_PAGES),
    ("negative", W.WI_DEV_BAD_SLOT), ("overflow", W.WI_DEV_BAD_SLOT), ("stack", W.WI_DEV_BAD_PAGE),
])
def test_plan_that_does_not_fit_changes_nothing(what, flag):
    have, new, capacity = [20, 5, 0], [30, 1, 2000], 2031
    table = make_table(have, 16, 140, 126, 6)
    if what == "pages":
        table.n_free.fill_(126)         # 2 + 125 are needed
    elif what == "capacity":
        capacity = 2030
    elif what == "row":
        table.block_table = table.block_table[:, :124].contiguous()
    elif what == "negative":
        new = [30, -1, 2000]
    elif what == "overflow":
        new = [30, 1, 2 ** 31 - 1]
        table.seq_lens[2] = 1
    elif what == "stack":
        table.n_free.fill_(table.free_pages.numel() + 1)
    before = (table.block_table.tolist(), table.seq_lens.tolist(), int(table.n_free))
    ws = W.serve_workspace(DEV)
    p = W.plan_pages(table, i32(new), capacity, update=True, ws=ws)
    assert W.read_device_status(ws) & flag
    assert (table.block_table.tolist(), table.seq_lens.tolist(), int(table.n_free)) == before
    assert set(p.slot_map.tolist()) == set(p.positions.tolist()) == {-1}
    assert p.starts.tolist() == [0] * 4
    # and the workspace serves the next step
    if what == "capacity":
        check_plan(table, new, 2031, ws=ws)
        assert W.read_device_status(ws) == 0


def test_plan_page_outside_the_pool():
    table = make_table([16, 16], 16, 20, 8, 7)
    table.free_pages[int(table.n_free) - 1] = 20       # request 0's first new page
    table.block_table[1, 0] = -3                       # a full page: not read
    ws = W.serve_workspace(DEV)
    p = check_plan(table, [17, 1], 18, ws=ws)
    assert p.slot_map.tolist()[:16] == [-1] * 16 and min(p.slot_map.tolist()[16:]) >= 0
    assert W.read_device_status(ws) == W.WI_DEV_BAD_PAGE


@pytest.mark.parametrize("left", [0, 1, 255])
def test_plans_of_many_tokens_in_place_keep_nothing_in_the_workspace(left):
    """Plans of 1 to 12 blocks on one workspace, whatever an ended call left
    behind the status word: the lengths advance and the workspace stays."""
    table = make_table([0] * 5, 16, 3000, 800, 61)
    ws = W.workspace(512, DEV)
    ws[4:].fill_(left)
    for new in ([1000, 17, 2000, 0, 5], [1] * 5, [3000, 3000, 1, 1, 6000], [400, 0, 0, 0, 625], [0, 0, 0, 1024, 1]):
        before = table.seq_lens.tolist()
        check_plan(table, new, sum(new) + 3, update=True, ws=ws)
        assert table.seq_lens.tolist() == [h + n for h, n in zip(before, new)]
        assert (ws[4:] == left).all()
    check_plan(table, [1, 2, 3, 4, 5000], 5000, update=True, ws=ws)     # over the capacity: as it was
    assert W.read_device_status(ws) == W.WI_DEV_NO_PAGES


def test_plan_in_place_of_one_of_the_two():
    for keep in ("seq_lens", "n_free"):
        table = make_table([9, 0], 16, 400, 200, 63)
        out = W.PagePlan.empty(table, 2600)
        setattr(out, keep, getattr(table, keep))
        check_plan(table, [2500, 99], 2600, out=out)


def test_plan_of_many_tokens_captured_in_place():
    table = make_table([30, 0, 17], 16, 900, 400, 65)
    new = i32([700, 0, 600])
    plan = W.PagePlan.empty(table, 1300, update=True)
    ws = W.serve_workspace(DEV)
    ref_table = table.block_table.tolist()
    lens, stack, n_free = table.seq_lens.tolist(), table.free_pages.tolist(), int(table.n_free)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        W.plan_pages(table, new, 1300, out=plan, update=True, ws=ws)
    for _ in range(4):
        ref_table, slots, _, _, lens, n_free = S.plan_reference(
            ref_table, lens, [700, 0, 600], stack, n_free, 16, 900, 1300)
        g.replay()
        assert plan.slot_map.tolist() == slots
        assert table.seq_lens.tolist() == lens and int(table.n_free) == n_free
    assert table.block_table.tolist() == ref_table


@pytest.mark.parametrize("new", [3, 4])
def test_plan_behind_the_last_tokens_an_int_counts(new):
    """A page in use whose end is position 2^31 - 1 (the table names one page
    again and again: a request may be longer than the pool)."""
    have, page = 2 ** 31 - 5, 16
    bt = torch.zeros(1, 2 ** 27, dtype=torch.int32, device=DEV)
    bt[0, -1] = 7
    table = W.PageTable(bt, i32([have]), i32([3, 2, 1]), i32([3]), page, 20)
    ws = W.serve_workspace(DEV)
    plan = W.plan_pages(table, i32([new]), 6, ws=ws)
    assert W.read_device_status(ws) == 0
    assert plan.slot_map.tolist() == [7 * 16 + 11 + i for i in range(new)] + [-1] * (6 - new)
    assert plan.positions.tolist() == [have + i for i in range(new)] + [-1] * (6 - new)
    assert plan.seq_lens.tolist() == [have + new] and int(plan.n_free) == 3
    # one more token does not fit an int
    W.plan_pages(table, i32([5]), 6, ws=ws)
    assert W.read_device_status(ws) == W.WI_DEV_BAD_SLOT


def test_plan_of_as_many_pages_as_an_int_counts():
    n = 2 ** 31 - 1
    table = W.PageTable.empty(1, n, 1, n, DEV)
    ws = W.serve_workspace(DEV)
    plan = W.plan_pages(table, i32([n]), n, ws=ws)
    assert W.read_device_status(ws) == 0
    assert plan.starts.tolist() == [0, n] and plan.seq_lens.tolist() == [n] and int(plan.n_free) == 0
    step = 1 << 28
    for i in range(0, n, step):
        want = torch.arange(i, min(n, i + step), dtype=torch.int32, device=DEV)
        for got in (plan.slot_map, plan.positions, table.block_table[0]):
            assert torch.equal(got[i:i + step], want)


# ---------------------------------------------------------------- appends

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,d,page,n", [(1, 64, 1, 1), (8, 128, 16, 37), (3, 64, 64, 300), (2, 128, 8, 4099)])
@pytest.mark.parametrize("fused", [False, True])
def test_append(dtype, H, d, page, n, fused):
    g = torch.Generator(device=DEV).manual_seed(n)
    n_pages = n // page + 7
    rows = torch.randn(n, 2 * H * d + (3 * H * d if fused else 0), generator=g, device=DEV).to(dtype)
    k = rows[:, -2 * H * d:-H * d].view(n, H, d)
    v = rows[:, -H * d:].view(n, H, d)
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    slots = torch.randperm(n_pages * page, generator=g, device=DEV)[:n].to(torch.int32)
    slots[::5] = -1
    pools = torch.randn(2, n_pages, H, page, d, generator=g, device=DEV).to(dtype)
    want = pools.clone()
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            want[0, s // page, :, s % page], want[1, s // page, :, s % page] = k[i], v[i]
    ws = W.serve_workspace(DEV)
    W.append_kv(k, v, slots, pools[0], pools[1], ws=ws)
    assert torch.equal(pools, want) and W.read_device_status(ws) == 0


def test_append_slot_outside_the_pool_is_skipped():
    pools = torch.zeros(2, 4, 2, 16, 64, device=DEV)
    k = torch.ones(3, 2, 64, device=DEV)
    ws = W.serve_workspace(DEV)
    W.append_kv(k, k, i32([64, 5, 2 ** 31 - 1]), pools[0], pools[1], ws=ws)
    assert W.read_device_status(ws) == W.WI_DEV_BAD_SLOT
    assert pools.sum() == 2 * 2 * 64 and (pools[:, 0, :, 5] == 1).all()
    W.append_kv(k[:0], k[:0], i32([]), pools[0], pools[1], ws=ws)


def test_without_a_workspace_a_call_tells_what_is_wrong():
    table = make_table([20, 5], 16, 8, 8, 67)
    table.n_free.fill_(0)
    before = table.block_table.clone()
    with pytest.raises(W.WaveIndexError, match="wi_plan_pages .WI_DEV_NO_PAGES") as e:
        W.plan_pages(table, i32([30, 1]), 40, update=True)
    assert e.value.status == W.WI_ERR_DEVICE_CHECK and torch.equal(table.block_table, before)
    pools, k = torch.zeros(2, 4, 2, 16, 64, device=DEV), torch.ones(3, 2, 64, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side):
        with pytest.raises(W.WaveIndexError, match="WI_DEV_BAD_SLOT"):
            W.append_kv(k, k, i32([64, 5, -1]), pools[0], pools[1], stream=stream)
        kv = W.KVCache(pools[0], pools[1], i32([[0, 4]]), [20])
        q = torch.zeros(1, 2, 64, device=DEV)
        torch.cuda.synchronize()
        with pytest.raises(W.WaveIndexError, match="wi_attend .WI_DEV_BAD_PAGE"):
            W.attend(q, kv, W.AttendParams(2, [1]), stream=stream)
    kv.block_table[0, 1] = 3
    W.attend(q, kv, W.AttendParams(2, [1]))
    # captured, nothing has run that could be told
    g = torch.cuda.CUDAGraph()
    slots = i32([7, 8, 9])
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        W.append_kv(k, k, slots, pools[0], pools[1])
        W.attend(q, kv, W.AttendParams(2, [1]))
    g.replay()
    torch.cuda.synchronize()
    assert (pools[:, 0, :, 7:10] == 1).all()


# -------------------------------------------------------------- attention

def make_cache(lens, H, d, page, dtype, seed, stale=float("nan"), spread=1.0):
    """A shuffled paged cache; every pool row that no token has is `stale`."""
    g = torch.Generator().manual_seed(seed)
    bt, n_pages = S.random_table(lens, page, seed)
    pools = torch.full((2, n_pages, H, page, d), stale, dtype=dtype)
    for b, T in enumerate(lens):
        pos = torch.arange(T)
        pages = bt[b].long()[pos // page]
        pools[0, pages, :, pos % page] = (spread * torch.randn(T, H, d, generator=g)).to(dtype)
        pools[1, pages, :, pos % page] = torch.randn(T, H, d, generator=g).to(dtype)
    pools = pools.to(DEV)
    return W.KVCache(pools[0], pools[1], bt.to(DEV), list(lens))


def make_q(n, Hq, d, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed + 1000)
    return (spread * torch.randn(n, Hq, d, generator=g)).to(dtype).to(DEV)


def check_attend(kv, q, q_lens, **kw):
    lens = kv.seq_lens
    q_lens = lens if q_lens is None else q_lens
    params = W.AttendParams(q.shape[1], q_lens)
    ws = kw.pop("ws", None)
    ws = W.attend_workspace(kv, params) if ws is None else ws
    out, lse = W.attend(q, kv, params, ws=ws, **kw)
    torch.cuda.synchronize()
    assert W.read_device_status(ws) == 0
    ref = S.attend_reference(q, kv.k_pool, kv.v_pool, kv.block_table, lens, q_lens)
    S.assert_attend(out, lse, ref, q.dtype, max(lens), q.shape[2])
    return out, lse


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_attend_ragged_prompts(dtype, d, G):
    kv = make_cache([1, 17, 130, 64, 300, 257], 2, d, 16, dtype, G)
    check_attend(kv, make_q(769, 2 * G, d, dtype, G), None)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [1, 2, 4, 8, 32, 128, 1024])
def test_attend_page_sizes(dtype, page):
    kv = make_cache([333, 40, 129], 2, 128, page, dtype, page)
    check_attend(kv, make_q(333 + 7, 4, 128, dtype, 1), [333, 0, 7])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,q_lens", [
    ([1], [1]), ([128], [1]), ([129], [1]), ([5000], [1]), ([3000, 1, 777], [1, 1, 1]),
    ([2500], [3]), ([2500, 900], [33, 900]), ([1025, 1024, 1023], [65, 64, 63]),
    ([600, 600, 600], [0, 600, 0]), ([4000, 200], [0, 1]), ([0, 70, 0], [0, 70, 0]),
    ([0, 1700, 0, 3], [0, 1, 0, 1]),
])
@pytest.mark.parametrize("H,G,d", [(1, 8, 128), (2, 1, 64), (4, 4, 128)])
def test_attend_chunks_and_single_tokens(dtype, lens, q_lens, H, G, d):
    kv = make_cache(lens, H, d, 16, dtype, sum(lens))
    check_attend(kv, make_q(sum(q_lens), H * G, d, dtype, 2), q_lens)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("q_len", [1, 260])
def test_attend_large_scores_rising_along_the_keys(dtype, q_len):
    """Scores over hundreds: a weight is 0 or all of it, and the running
    maximum rises again and again."""
    kv = make_cache([900], 1, 64, 16, dtype, 9, spread=6.0)
    pages = kv.block_table[0].long()[torch.arange(900, device=DEV) // 16]
    ramp = torch.linspace(0.1, 3.0, 900, device=DEV)[:, None, None]
    rows = torch.arange(900, device=DEV) % 16
    kv.k_pool[pages, :, rows] = (kv.k_pool[pages, :, rows].float().abs() * ramp).to(dtype)
    check_attend(kv, make_q(q_len, 4, 64, dtype, 3, spread=3.0).abs(), [q_len])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_strided_rows_and_rows_behind_the_last_sequence(dtype):
    lens, H, G, d, n = [70, 333], 2, 4, 128, 403
    kv = make_cache(lens, H, d, 16, dtype, 11)
    wide = make_q(n + 9, H * G + 2 * H, d, dtype, 4)
    q = wide[:, :H * G]
    into = torch.full((n + 9, H * G + 3, d), 7.0, dtype=dtype, device=DEV)
    lse = torch.full((n + 9, H * G), 7.0, device=DEV)
    out, _ = check_attend(kv, q, None, out=into[:, 2:2 + H * G], lse=lse)
    assert (into[n:] == 7).all() and (into[:, :2] == 7).all() and (into[:, -1] == 7).all()
    assert (lse[n:] == 7).all()
    plain, _ = W.attend(q[:n].contiguous(), kv, W.AttendParams(H * G))
    assert torch.equal(plain, out[:n])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("lens,q_lens", [([300], [300]), ([1500], [40])])
def test_attend_later_keys_have_no_effect(dtype, bad, lens, q_lens):
    """A key or value that is not finite reaches the queries behind it, and
    only those."""
    T, n = lens[0], q_lens[0]
    kv = make_cache(lens, 2, 128, 16, dtype, 13)
    q = make_q(n, 8, 128, dtype, 5)
    clean, clean_lse = W.attend(q, kv, W.AttendParams(8, q_lens))
    at = T - n // 2                     # a position half way through the queries
    i = at - (T - n)
    page, row = int(kv.block_table[0, at // 16]), at % 16
    kv.v_pool[page, 0, row, 5] = bad
    kv.k_pool[page, 1, row, :] = bad
    out, lse = W.attend(q, kv, W.AttendParams(8, q_lens))
    assert torch.equal(out[:i], clean[:i]) and torch.equal(lse[:i], clean_lse[:i])
    hit = out[i:, :4, 5]
    assert (hit == bad).all() if bad == bad else torch.isnan(hit).all()
    rest = [c for c in range(128) if c != 5]
    assert torch.equal(out[:, :4, rest], clean[:, :4, rest])      # the other channels
    assert torch.equal(lse[:, :4], clean_lse[:, :4])
    if bad != bad:
        assert torch.isnan(out[i:, 4:]).all() and torch.isnan(lse[i:, 4:]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_page_outside_the_pool_is_flagged(dtype):
    kv = make_cache([300, 120], 2, 128, 16, dtype, 15)
    q = make_q(420, 4, 128, dtype, 6)
    params = W.AttendParams(4)
    ws = W.attend_workspace(kv, params)
    clean, _ = W.attend(q, kv, params, ws=ws)
    for wrong in (-1, kv.k_pool.shape[0], 2 ** 31 - 1):
        kv.block_table[0, 18] = wrong              # positions 288..299
        out, _ = W.attend(q, kv, params, ws=ws)
        assert W.read_device_status(ws) == W.WI_DEV_BAD_PAGE
        assert torch.equal(out[:288], clean[:288]) and torch.equal(out[300:], clean[300:])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_repeats_bit_for_bit_on_a_used_workspace(dtype):
    kv = make_cache([5000, 310], 2, 128, 16, dtype, 17)
    q = make_q(2, 8, 128, dtype, 7)
    params = W.AttendParams(8, [1, 1])
    first, first_lse = check_attend(kv, q, [1, 1])
    big = W.workspace(1 << 24, DEV)
    big[256:].fill_(255)                           # what another call left
    for _ in range(2):
        out, lse = W.attend(q, kv, params, ws=big)
        assert torch.equal(out, first) and torch.equal(lse, first_lse)


def test_attend_on_another_stream_and_captured():
    kv = make_cache([2000, 77], 2, 128, 16, BF16, 19)
    params = W.AttendParams(8, [1, 77])
    q = make_q(78, 8, 128, BF16, 8)
    ref, ref_lse = check_attend(kv, q, [1, 77])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = W.attend(q, kv, params, stream=side)
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    ws, into, into_lse = W.attend_workspace(kv, params), torch.zeros_like(ref), torch.zeros_like(ref_lse)
    held = q.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        W.attend(held, kv, params, out=into, lse=into_lse, ws=ws)
    for seed in (8, 9):
        held.copy_(make_q(78, 8, 128, BF16, seed))
        g.replay()
        want, want_lse = W.attend(held, kv, params)
        assert torch.equal(into, want) and torch.equal(into_lse, want_lse)
    with pytest.raises(W.WaveIndexError):
        W.attend(q, kv, params, ws=W.workspace(256, DEV))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [1, 2, 4, 8, 64, 1024])
@pytest.mark.parametrize("G,q_lens", [(1, [16, 1, 9]), (8, [2, 1, 0]), (4, [4, 3, 1])])
def test_attend_few_rows_page_sizes(dtype, page, G, q_lens):
    """Blocks of at most 16 rows, full ones among them."""
    kv = make_cache([1300, 128, 333], 2, 128, page, dtype, page + G)
    check_attend(kv, make_q(sum(q_lens), 2 * G, 128, dtype, page), q_lens)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 15, 16, 17, 127, 128, 129, 255, 257])
def test_attend_one_token_at_every_edge_of_a_tile(dtype, d, T):
    kv = make_cache([T, T + 1000], 2, d, 16, dtype, T)
    check_attend(kv, make_q(2, 4, d, dtype, T), [1, 1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T", [40, 1500, 1536])
def test_attend_later_keys_have_no_effect_on_few_rows(dtype, bad, T):
    kv = make_cache([T], 2, 64, 16, dtype, 21)
    q = make_q(6, 4, 64, dtype, 21)
    clean, clean_lse = W.attend(q, kv, W.AttendParams(4, [6]))
    at = T - 3
    page, row = int(kv.block_table[0, at // 16]), at % 16
    kv.v_pool[page, 0, row, 5] = bad
    kv.k_pool[page, 1, row] = float("nan")
    out, lse = W.attend(q, kv, W.AttendParams(4, [6]))
    assert torch.equal(out[:3], clean[:3]) and torch.equal(lse[:3], clean_lse[:3])
    hit = out[3:, :2, 5]
    assert (hit == bad).all() if bad == bad else torch.isnan(hit).all()
    assert torch.equal(out[:, :2, 6:], clean[:, :2, 6:]) and torch.equal(lse[:, :2], clean_lse[:, :2])
    assert torch.isnan(out[3:, 2:]).all() and torch.isnan(lse[3:, 2:]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_full_batch(dtype):
    rng = np.random.default_rng(23)
    lens = rng.integers(1, 260, 256).tolist()
    q_lens = [int(rng.integers(0, min(T, 40) + 1)) for T in lens]
    kv = make_cache(lens, 1, 64, 16, dtype, 23)
    check_attend(kv, make_q(sum(q_lens), 2, 64, dtype, 23), q_lens)
    check_attend(kv, make_q(256, 2, 64, dtype, 24), [1] * 256)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_offsets_past_32_bits(dtype):
    """A pool of more than 2^32 elements: rows appended to and attended on its
    last pages."""
    H, page, d, lens = 8, 16, 128, [700, 33]
    n_pages = 2 ** 32 // (H * page * d) + 64
    pools = torch.empty(2, n_pages, H, page, d, dtype=dtype, device=DEV)
    need = [-(-T // page) for T in lens]
    bt = torch.full((2, max(need)), -1, dtype=torch.int32)
    last = torch.arange(n_pages - sum(need), n_pages, dtype=torch.int32).flip(0)
    bt[0], bt[1, :need[1]] = last[:need[0]], last[need[0]:]
    kv = W.KVCache(pools[0], pools[1], bt.to(DEV), lens)
    k, v = make_q(sum(lens), H, d, dtype, 50), make_q(sum(lens), H, d, dtype, 51)
    pos = torch.cat([torch.arange(T) for T in lens])
    req = torch.repeat_interleave(torch.arange(2), torch.tensor(lens))
    slots = (bt[req, pos // page] * page + pos % page).to(torch.int32).to(DEV)
    W.append_kv(k, v, slots, pools[0], pools[1])
    # the same rows in a small pool
    small = torch.zeros(2, sum(need), H, page, d, dtype=dtype, device=DEV)
    tail = int(n_pages - sum(need))
    for q_lens in ([5, 33], [1, 1]):
        q = make_q(sum(q_lens), 16, d, dtype, 52)
        out, lse = W.attend(q, kv, W.AttendParams(16, q_lens))
        small.copy_(pools[:, tail:])
        near = W.KVCache(small[0], small[1], torch.where(bt >= 0, bt - tail, bt).to(DEV), lens)
        want, want_lse = W.attend(q, near, W.AttendParams(16, q_lens))
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert torch.equal(pools[0, int(bt[0, 3]), :, 7], k[3 * page + 7])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_captured_single_tokens_share_a_workspace(dtype):
    """Two graphs of split calls of other sizes on one workspace, replayed in
    turns."""
    caches = [make_cache([6000, 800], 2, 128, 16, dtype, 25), make_cache([300, 9000, 5], 2, 128, 16, dtype, 26)]
    params = [W.AttendParams(8, [1, 1]), W.AttendParams(8, [1, 1, 1])]
    ws = W.workspace(max(W.attend_workspace_bytes(c, p) for c, p in zip(caches, params)), DEV)
    ws[256:].fill_(255)
    graphs, outs = [], []
    for i, (kv, p) in enumerate(zip(caches, params)):
        q = make_q(len(kv.seq_lens), 8, 128, dtype, 27 + i)
        want = W.attend(q, kv, p)
        into = [torch.zeros_like(x) for x in want]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            W.attend(q, kv, p, out=into[0], lse=into[1], ws=ws)
        graphs.append((g, q))
        outs.append((want, into))
    for _ in range(3):
        for (g, _), (want, into) in zip(graphs, outs):
            into[0].zero_()
            g.replay()
            assert torch.equal(into[0], want[0]) and torch.equal(into[1], want[1])


def test_plan_and_append_on_another_stream():
    side = torch.cuda.Stream()
    table = make_table([30, 0, 17], 16, 40, 8, 27)
    pools = torch.zeros(2, 40, 2, 16, 64, device=DEV)
    k = torch.randn(6, 2, 64, device=DEV)
    torch.cuda.synchronize()
    plan = W.plan_pages(table, i32([3, 1, 2]), 6, update=True, stream=side)
    W.append_kv(k, 2 * k, plan.slot_map, pools[0], pools[1], stream=side)
    side.synchronize()
    assert table.seq_lens.tolist() == [33, 1, 19]
    for i, s in enumerate(plan.slot_map.tolist()):
        assert torch.equal(pools[0, s // 16, :, s % 16], k[i])
        assert torch.equal(pools[1, s // 16, :, s % 16], 2 * k[i])


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_tensors_on_another_device_than_the_current_one():
    kv0 = make_cache([500, 3], 2, 64, 16, BF16, 29)
    q = make_q(503, 4, 64, BF16, 29)
    want, _ = W.attend(q, kv0, W.AttendParams(4))
    kv1 = W.KVCache(*(x.to("cuda:1") for x in (kv0.k_pool, kv0.v_pool, kv0.block_table)), [500, 3])
    out, _ = W.attend(q.to("cuda:1"), kv1, W.AttendParams(4))
    assert out.device.index == 1 and torch.equal(out.to(DEV), want)


# A weight as two bf16 parts: the second is the rest of the first, off by half
# a step of itself, so by 2^-8 * 2^-8 of the weight.
TWO_PARTS = S.U[BF16] ** 2


@pytest.mark.parametrize("lens,q_lens,H,G,d", [
    ([2], [1], 4, 8, 128), ([3, 5], [1, 2], 4, 8, 64), ([18], [16], 4, 1, 128), ([1500, 4], [2, 2], 2, 8, 128),
])
def test_attend_few_rows_keep_16_bits_of_a_weight(lens, q_lens, H, G, d):
    """Few keys of about equal weight: where the values nearly cancel, a weight
    rounded to bf16 is many times the bound."""
    kv = make_cache(lens, H, d, 16, BF16, 31, spread=0.3)
    q = make_q(sum(q_lens), H * G, d, BF16, 31)
    out, lse = W.attend(q, kv, W.AttendParams(H * G, q_lens))
    ref = S.attend_reference(q, kv.k_pool, kv.v_pool, kv.block_table, lens, q_lens)
    S.assert_attend(out, lse, ref, BF16, max(lens), d, TWO_PARTS)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("T,n,G", [(300, 1, 4), (1500, 3, 4), (1500, 12, 1), (700, 40, 4)])
def test_attend_value_that_is_not_finite_and_all_see(dtype, bad, T, n, G):
    kv = make_cache([T], 2, 128, 16, dtype, 35, spread=0.3)
    q = make_q(n, 2 * G, 128, dtype, 35)
    clean, clean_lse = W.attend(q, kv, W.AttendParams(2 * G, [n]))
    for at in (3, T // 2):
        kv.v_pool[int(kv.block_table[0, at // 16]), 1, at % 16, 7] = bad
    kv.v_pool[int(kv.block_table[0, 0]), 1, 4, 9] = -bad
    out, lse = W.attend(q, kv, W.AttendParams(2 * G, [n]))
    assert torch.equal(lse, clean_lse) and torch.equal(out[:, :G], clean[:, :G])
    for c, want in ((7, bad), (9, -bad)):
        hit = out[:, G:, c]
        assert (hit == want).all() if bad == bad else torch.isnan(hit).all()
    rest = [c for c in range(128) if c not in (7, 9)]
    assert torch.equal(out[:, G:, rest], clean[:, G:, rest])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,q_lens,H,G", [
    ([20], [20], 2, 1), ([5, 40], [5, 17], 2, 4), ([300], [300], 1, 1), ([130, 0, 9], [70, 0, 9], 2, 8),
    ([2600], [70], 1, 4), ([700, 690], [1, 300], 2, 2),
])
def test_attend_exact_weights(d, lens, q_lens, H, G):
    """16 bits of a weight at the caller's wish: queries with few keys of about
    equal weight, blocks of 128 and 256 rows, split and not."""
    kv = make_cache(lens, H, d, 16, BF16, 37, spread=0.3)
    q = make_q(sum(q_lens), H * G, d, BF16, 37)
    out, lse = W.attend(q, kv, W.AttendParams(H * G, q_lens, exact_weights=True))
    ref = S.attend_reference(q, kv.k_pool, kv.v_pool, kv.block_table, lens, q_lens)
    S.assert_attend(out, lse, ref, BF16, max(lens), d, TWO_PARTS)
    other, other_lse = W.attend(q, kv, W.AttendParams(H * G, q_lens))
    assert torch.equal(other_lse, lse)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("T,n", [(300, 300), (1500, 40), (900, 70)])
def test_attend_exact_weights_with_values_that_are_not_finite(bad, T, n):
    kv = make_cache([T], 2, 128, 16, BF16, 39, spread=0.3)
    q, prm = make_q(n, 8, 128, BF16, 39), W.AttendParams(8, [n], exact_weights=True)
    clean, clean_lse = W.attend(q, kv, prm)
    late = T - n // 2                      # half of the queries see it, and all see key 3 but a prompt's first
    for at, c in ((3, 7), (late, 9)):
        kv.v_pool[int(kv.block_table[0, at // 16]), 1, at % 16, c] = bad
    out, lse = W.attend(q, kv, prm)
    assert torch.equal(lse, clean_lse) and torch.equal(out[:, :4], clean[:, :4])
    for at, c in ((3, 7), (late, 9)):
        i = max(0, at - (T - n))
        assert torch.equal(out[:i, :, c], clean[:i, :, c])
        hit = out[i:, 4:, c]
        assert (hit == bad).all() if bad == bad else torch.isnan(hit).all()
    rest = [c for c in range(128) if c not in (7, 9)]
    assert torch.equal(out[:, 4:, rest], clean[:, 4:, rest])


def steps_cache(T, d, dtype, seed, rise):
    """Scores 0 and `rise` (base 2) in turns of 128 keys for a query of ones in
    channel 0: a maximum that a block meets late."""
    kv = make_cache([T], 1, d, 16, dtype, seed)
    pos = torch.arange(T, device=DEV)
    pages, rows = kv.block_table[0].long()[pos // 16], pos % 16
    k = torch.zeros(T, 1, d, device=DEV)
    k[:, 0, 0] = torch.where(pos % 256 < 128, 0.0, rise * math.sqrt(d) * math.log(2))
    kv.k_pool[pages, :, rows] = k.to(dtype)
    return kv


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("q_len", [1, 4, 20, 260])
@pytest.mark.parametrize("rise", [22, 40])
@pytest.mark.parametrize("exact", [False, True])
def test_attend_range_of_values(dtype, q_len, rise, exact):
    """Values up to 2^114 (900 of them stay below 2^127) and down to 2^-90."""
    T, d, G = 900, 64, 4
    kv = steps_cache(T, d, dtype, 33, rise)
    q = torch.zeros(q_len, G, d, device=DEV)
    q[:, :, 0] = 1
    q, prm = q.to(dtype), W.AttendParams(G, [q_len], exact_weights=exact)
    ref = S.attend_reference(q, kv.k_pool, kv.v_pool, kv.block_table, [T], [q_len])
    v = kv.v_pool.clone()
    for power in (112, -90):
        kv.v_pool.copy_((v.double() * 2.0 ** power).to(dtype))
        out, lse = W.attend(q, kv, prm)
        S.assert_attend(out.double() * 2.0 ** -power, lse, ref, dtype, T, d)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_workspace_of_the_bound_serves_all_steps(dtype):
    """Growing contexts, chunks and single tokens, sequences that come and go."""
    H, G, d, page, top, most = 2, 4, 128, 16, 6000, 70
    kv = make_cache([top, top, 900], H, d, page, dtype, 41)
    ws = W.workspace(W.attend_workspace_bound(kv, H * G, top, most), DEV)
    for lens, q_lens in (([70, 70, 0], [70, 70, 0]), ([513, 600, 0], [70, 1, 0]), ([4366, 30, 900], [1, 30, 1]),
                         ([4657, 31, 0], [1, 1, 0]), ([6000, 6000, 900], [1, 1, 1]), ([6000, 5000, 2], [70, 3, 2])):
        step = W.KVCache(kv.k_pool, kv.v_pool, kv.block_table, lens)
        check_attend(step, make_q(sum(q_lens), H * G, d, dtype, sum(lens)), q_lens, ws=ws)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("batch,T,n,H,G", [(24, 4096, 1, 1, 8), (40, 3000, 2, 2, 1), (24, 2300, 17, 1, 8)])
def test_attend_splits_keys_of_more_than_16_sequences(dtype, batch, T, n, H, G):
    """Both joins (2720 rows, of 20 sequences with queries, are many) behind the kernels of
    large batches."""
    lens = [T - 37 * (b % 5) for b in range(batch)]
    q_lens = [n if b % 7 else 0 for b in range(batch)]
    kv = make_cache(lens, H, 128, 16, dtype, batch)
    assert W.attend_workspace_bytes(kv, W.AttendParams(H * G, q_lens)) > 256
    check_attend(kv, make_q(sum(q_lens), H * G, 128, dtype, batch), q_lens)


@pytest.mark.parametrize("dtype,T,d,n", [(BF16, 131072, 128, 1), (BF16, 131000, 64, 1), (BF16, 131072, 128, 17),
                                         (F32, 40000, 128, 1), (F32, 79999, 64, 1)])
def test_attend_of_more_than_128_runs(dtype, T, d, n):
    """A join of more parts than one round of its four warps takes."""
    kv = make_cache([T], 1, d, 16, dtype, 43)
    size = W.attend_workspace_bytes(kv, W.AttendParams(1, [n]))
    assert size > 256 + 128 * n * (8 + 4 * d)
    check_attend(kv, make_q(n, 1, d, dtype, 43), [n])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_output_beside_the_queries_in_one_row(dtype):
    kv = make_cache([70, 90], 2, 64, 16, dtype, 45)
    wide = make_q(160, 17, 64, dtype, 45)
    q = wide[:, 1:9].clone()
    want, _ = W.attend(q, kv, W.AttendParams(8))
    for first in (9, 0):
        rows = wide.clone()
        at = 1 if first else 8
        rows[:, at:at + 8] = q
        out = rows[:, first:first + 8]
        W.attend(rows[:, at:at + 8], kv, W.AttendParams(8), out=out)
        assert torch.equal(out, want) and torch.equal(rows[:, at:at + 8], q)
    with pytest.raises(W.WaveIndexError):
        W.attend(wide[:, 1:9], kv, W.AttendParams(8), out=wide[:, 2:10])


@pytest.mark.parametrize("dtype,n", [(BF16, 1), (BF16, 3), (F32, 1)])
def test_attend_over_the_longest_sequence(dtype, n):
    """2^31 - 256 tokens on three pages named again and again: equal scores and
    values of one, so each query's output is one and its mass a count."""
    T, page, G = 2 ** 31 - 256, 1024, 8
    k, v = torch.zeros(3, 1, page, 64, dtype=dtype, device=DEV), torch.ones(3, 1, page, 64, dtype=dtype, device=DEV)
    bt = (torch.arange(2 ** 21, device=DEV) % 3).to(torch.int32)[None]
    kv = W.KVCache(k, v, bt, [T])
    out, lse = W.attend(make_q(n, G, 64, dtype, 47), kv, W.AttendParams(G, [n]))
    assert (out == 1).all()
    seen = torch.arange(T - n + 1, T + 1, dtype=torch.float64, device=DEV)[:, None]
    assert ((lse.double() - seen.log()).abs() <= 2.0 ** -22 * 32).all()


def test_attend_calls_at_once_on_two_streams():
    """Split and whole calls side by side, each with a workspace of its own."""
    calls = []
    for seed, lens, q_lens, dtype in ((51, [9000, 300], [1, 1], BF16), (52, [2000, 700], [300, 700], BF16),
                                      (53, [5000], [40], BF16), (54, [3000, 20], [1, 20], F32)):
        kv, prm = make_cache(lens, 2, 128, 16, dtype, seed), W.AttendParams(8, q_lens)
        q = make_q(sum(q_lens), 8, 128, dtype, seed)
        ws = W.attend_workspace(kv, prm)
        calls.append((q, kv, prm, ws, W.attend(q, kv, prm, ws=ws)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for i in range(40):
        q, kv, prm, ws, _ = calls[2 * (i // 2 % 2) + i % 2]     # (a workspace stays on one stream)
        got.append(W.attend(q, kv, prm, ws=ws, stream=streams[i % 2]))
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        want, want_lse = calls[2 * (i // 2 % 2) + i % 2][4]
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("n,exact", [(1, False), (20, False), (260, False), (260, True)])
@pytest.mark.parametrize("gap", [90, 110, 140])
def test_attend_infinite_value_of_a_small_weight(n, exact, gap):
    """An infinity under a weight of 2^-gap of the largest is infinite, not 0
    times it."""
    T, d, G = 900, 64, 4
    kv = steps_cache(T, d, BF16, 55, gap)
    q = torch.zeros(n, G, d, dtype=BF16, device=DEV)
    q[:, :, 0] = 1
    prm = W.AttendParams(G, [n], exact_weights=exact)
    clean, _ = W.attend(q, kv, prm)
    for at, c in ((5, 3), (300, 8)):            # keys of score 0
        kv.v_pool[int(kv.block_table[0, at // 16]), 0, at % 16, c] = math.inf
    out, lse = W.attend(q, kv, prm)
    assert torch.isfinite(lse).all() and (out[:, :, 3] == math.inf).all() and (out[:, :, 8] == math.inf).all()
    rest = [c for c in range(d) if c not in (3, 8)]
    assert torch.equal(out[:, :, rest], clean[:, :, rest])


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_to_decode_through_one_cache(dtype):
    """Pages planned, a prompt's rows appended and attended, decode steps
    planned, appended and attended, then the index built from the same cache:
    its decode with every cluster retrieved is the same dense attention."""
    H, G, d, page, lens = 2, 4, 128, 16, [700, 33, 260]
    B, Hq = len(lens), H * G
    n_pages, max_pages = 80, 60
    table = W.PageTable.empty(B, max_pages, page, n_pages, DEV)
    pools = torch.full((2, n_pages, H, page, d), float("nan"), dtype=dtype, device=DEV)
    ws = W.serve_workspace(DEV)
    have = [0] * B
    for step, new in enumerate(([700, 20, 260], [0, 13, 0], [1, 1, 1], [1, 0, 1], [1, 1, 1])):
        n = sum(new)
        rows = make_q(n, Hq + 2 * H, d, dtype, 40 + step)
        q, k, v = rows[:, :Hq], rows[:, Hq:Hq + H], rows[:, Hq + H:]
        plan = W.plan_pages(table, i32(new), n, update=True, ws=ws)
        W.append_kv(k, v, plan.slot_map, pools[0], pools[1], ws=ws)
        have = [h + m for h, m in zip(have, new)]
        assert table.seq_lens.tolist() == have
        kv = W.KVCache(pools[0], pools[1], table.block_table, have)
        # the rows are where the table says they are
        for b in range(B):
            for i in range(new[b]):
                pos, t = have[b] - new[b] + i, int(plan.starts[b]) + i
                if i in (0, new[b] - 1):
                    assert torch.equal(pools[0, int(table.block_table[b, pos // page]), :, pos % page], k[t])
        out, lse = check_attend(kv, q, new)
    assert W.read_device_status(ws) == 0
    idx = W.build_index(kv, 256, 16, 2)
    dp = W.DecodeParams(n_q_heads=Hq, n_sink=4, window=16, topk_clusters=10 ** 6)
    dec, dec_lse = W.decode(q.contiguous(), idx, dp)
    ref = S.attend_reference(q, kv.k_pool, kv.v_pool, kv.block_table, have, new)
    tol_out, tol_lse = S.attend_bounds(*ref, dtype, max(have), d)
    gap = (dec.double() - out.double()).abs().cpu().numpy()
    # decode's own bound against dense attention is 2e-4 (bf16) or 1e-5 (fp32) of rms / max
    assert (gap <= tol_out + 2e-4 * np.abs(ref[0]).max()).all()
    assert (np.abs(dec_lse.cpu().numpy() - lse.cpu().numpy()) <= tol_lse + 1e-4).all()
