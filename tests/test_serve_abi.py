"""Argument checks of the serving calls (no GPU: every refusal comes before
any CUDA call), the plan of the split key axis, and the plain page plan the
GPU tests compare with, by hand-counted cases."""
import ctypes as C

import pytest
import torch

import retrieval_sparse_attention_wave_b200 as W
from tests import serve_harness as S
from tests.test_abi import FAKE, kv_struct


def page_plan(**over):
    p = W.WiPagePlan(4, 16, 100, FAKE, FAKE + 0x1000, FAKE + 0x2000, 8, FAKE + 0x3000, 100,
                     FAKE + 0x4000, FAKE + 0x5000, FAKE + 0x6000, FAKE + 0x7000, 64, FAKE + 0x8000,
                     FAKE + 0x9000)
    for k, v in over.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over,expect", [
    (dict(batch=0), W.WI_ERR_INVALID_ARG),
    (dict(batch=257), W.WI_ERR_UNSUPPORTED),
    (dict(page_size=12), W.WI_ERR_INVALID_ARG),
    (dict(page_size=2048), W.WI_ERR_INVALID_ARG),
    (dict(n_pages=0), W.WI_ERR_INVALID_ARG),
    (dict(n_pages=2 ** 28), W.WI_ERR_UNSUPPORTED),    # slots pass 32 bits
    (dict(max_pages=0), W.WI_ERR_INVALID_ARG),
    (dict(capacity=-1), W.WI_ERR_INVALID_ARG),
    (dict(max_free=-1), W.WI_ERR_INVALID_ARG),
    (dict(seq_lens=None), W.WI_ERR_INVALID_ARG),
    (dict(new_lens=None), W.WI_ERR_INVALID_ARG),
    (dict(block_table=None), W.WI_ERR_INVALID_ARG),
    (dict(free_pages=None), W.WI_ERR_INVALID_ARG),
    (dict(n_free=None), W.WI_ERR_INVALID_ARG),
    (dict(seq_lens_out=None), W.WI_ERR_INVALID_ARG),
    (dict(n_free_out=None), W.WI_ERR_INVALID_ARG),
    (dict(starts=None), W.WI_ERR_INVALID_ARG),
    (dict(slot_map=None), W.WI_ERR_INVALID_ARG),
    (dict(slot_map=FAKE + 2), W.WI_ERR_INVALID_ARG),
    (dict(), W.WI_ERR_WORKSPACE),                     # all valid: the workspace is checked last
    (dict(positions=None, free_pages=None, max_free=0), W.WI_ERR_WORKSPACE),
])
def test_plan_pages_refusals(over, expect):
    assert W.lib().wi_plan_pages(C.byref(page_plan(**over)), FAKE, 255, None) == expect


def test_plan_pages_workspace():
    p = page_plan()
    assert W.lib().wi_plan_pages(C.byref(p), None, 256, None) == W.WI_ERR_WORKSPACE
    assert W.lib().wi_plan_pages(C.byref(p), FAKE + 16, 256, None) == W.WI_ERR_WORKSPACE
    assert W.lib().wi_plan_pages(None, FAKE, 256, None) == W.WI_ERR_INVALID_ARG


def kv_append(**over):
    a = W.WiKVAppend(W.WI_BF16, 5, 8, 128, 16, 100, FAKE, FAKE + 0x10000, 0, 0, FAKE + 0x20000,
                     FAKE + 0x30000, FAKE + 0x40000)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,expect", [
    (dict(dtype=3), W.WI_ERR_INVALID_ARG),
    (dict(n_tokens=-1), W.WI_ERR_INVALID_ARG),
    (dict(n_kv_heads=0), W.WI_ERR_INVALID_ARG),
    (dict(head_dim=96), W.WI_ERR_UNSUPPORTED),
    (dict(page_size=3), W.WI_ERR_INVALID_ARG),
    (dict(n_pages=0), W.WI_ERR_INVALID_ARG),
    (dict(n_pages=2 ** 30), W.WI_ERR_UNSUPPORTED),
    (dict(k=None), W.WI_ERR_INVALID_ARG),
    (dict(k=FAKE + 8), W.WI_ERR_INVALID_ARG),
    (dict(v_pool=None), W.WI_ERR_INVALID_ARG),
    (dict(v_pool=FAKE + 0x30000), W.WI_ERR_INVALID_ARG),     # one pool for keys and values
    (dict(slot_map=None), W.WI_ERR_INVALID_ARG),
    (dict(k_stride=1000), W.WI_ERR_INVALID_ARG),      # shorter than a token's row
    (dict(v_stride=1028), W.WI_ERR_INVALID_ARG),      # not a multiple of 16 bytes
    (dict(k_stride=1032), W.WI_ERR_WORKSPACE),
    (dict(), W.WI_ERR_WORKSPACE),
])
def test_append_kv_refusals(over, expect):
    assert W.lib().wi_append_kv(C.byref(kv_append(**over)), FAKE, 0, None) == expect


def test_append_of_nothing_is_ok():
    a = kv_append(n_tokens=0, k=None, v=None, slot_map=None)
    assert W.lib().wi_append_kv(C.byref(a), FAKE, 256, None) == W.WI_OK


def attend_params(n_q_heads=32, q_lens=None, **over):
    p = W.WiAttendParams(n_q_heads, None, 0, 0)
    if q_lens is not None:
        p._keep = (C.c_int32 * len(q_lens))(*q_lens)
        p.q_lens = C.cast(p._keep, C.POINTER(C.c_int32))
    for k, v in over.items():
        setattr(p, k, v)
    return p


def attend_size(kv, p):
    n = C.c_size_t()
    return W.lib().wi_attend_workspace_size(C.byref(kv), C.byref(p), C.byref(n)), n.value


@pytest.mark.parametrize("kv,p,expect", [
    (dict(), dict(), W.WI_OK),
    (dict(), dict(q_lens=[0]), W.WI_OK),
    (dict(), dict(q_lens=[4096]), W.WI_OK),
    (dict(), dict(q_lens=[4097]), W.WI_ERR_INVALID_ARG),
    (dict(), dict(q_lens=[-1]), W.WI_ERR_INVALID_ARG),
    (dict(), dict(n_q_heads=0), W.WI_ERR_INVALID_ARG),
    (dict(), dict(n_q_heads=12), W.WI_ERR_INVALID_ARG),
    (dict(), dict(n_q_heads=24), W.WI_ERR_UNSUPPORTED),      # G = 3
    (dict(), dict(n_q_heads=128), W.WI_ERR_UNSUPPORTED),     # G = 16
    (dict(), dict(q_stride=4095), W.WI_ERR_INVALID_ARG),
    (dict(), dict(out_stride=4100), W.WI_ERR_INVALID_ARG),
    (dict(), dict(q_stride=6144), W.WI_OK),
    (dict(seq=[0]), dict(), W.WI_OK),                        # an empty slot of a batch
    (dict(seq=[0]), dict(q_lens=[1]), W.WI_ERR_INVALID_ARG),
    (dict(seq=[-1]), dict(), W.WI_ERR_INVALID_ARG),
    (dict(seq=[70000]), dict(), W.WI_ERR_INVALID_ARG),       # more pages than the table's row
    (dict(head_dim=96), dict(), W.WI_ERR_UNSUPPORTED),
    (dict(n_pages=2 ** 25), dict(), W.WI_ERR_UNSUPPORTED),   # pool rows pass 32 bits
    (dict(k_pool=None), dict(), W.WI_ERR_INVALID_ARG),
])
def test_attend_refusals(kv, p, expect):
    assert attend_size(kv_struct(**kv), attend_params(**p))[0] == expect


@pytest.mark.parametrize("T,expect", [
    (2 ** 31 - 256, W.WI_OK), (2 ** 31 - 255, W.WI_ERR_UNSUPPORTED), (2 ** 31 - 1, W.WI_ERR_UNSUPPORTED),
])
@pytest.mark.parametrize("n", [1, 2000])
def test_attend_positions_fit_whole_tiles(T, n, expect):
    kv = kv_struct(seq=[T], n_kv_heads=1, page_size=1024, max_pages=2 ** 21)
    assert attend_size(kv, attend_params(8, q_lens=[n]))[0] == expect


def test_attend_rejects_before_any_cuda_call():
    lib, kv, p = W.lib(), kv_struct(), attend_params(q_lens=[1])
    st, need = attend_size(kv, p)
    assert st == W.WI_OK and need % 256 == 0
    call = lambda q, out, lse, ws, n: lib.wi_attend(q, C.byref(kv), C.byref(p), out, lse, ws, n, None)
    assert call(None, FAKE, None, FAKE, need) == W.WI_ERR_INVALID_ARG
    assert call(FAKE, None, None, FAKE, need) == W.WI_ERR_INVALID_ARG
    assert call(FAKE, FAKE, None, FAKE, need) == W.WI_ERR_INVALID_ARG          # out is q
    assert call(FAKE + 8, FAKE, None, FAKE, need) == W.WI_ERR_INVALID_ARG
    assert call(FAKE, FAKE + 0x100, FAKE + 2, FAKE, need) == W.WI_ERR_INVALID_ARG
    assert call(FAKE, FAKE + 0x100, None, None, need) == W.WI_ERR_WORKSPACE
    assert call(FAKE, FAKE + 0x100, None, FAKE, need - 1) == W.WI_ERR_WORKSPACE
    assert call(FAKE, FAKE + 0x100, None, FAKE + 16, need) == W.WI_ERR_WORKSPACE
    none = attend_params(q_lens=[0])
    assert lib.wi_attend(None, C.byref(kv), C.byref(none), None, None, FAKE, need, None) == W.WI_OK


@pytest.mark.parametrize("q,out,qs,os,n", [
    (0, 256, 0, 0, 1), (256, 0, 0, 0, 1), (0, 8176, 0, 0, 3), (8192, 16, 0, 0, 1),
    (0, 8192, 0, 0, 2),                  # the second row of q
    (16384 - 16, 0, 8192, 8192, 3),      # the last bytes of a row beside it
    (0, 8192, 6144, 6144, 2),            # 12288 bytes apart: its end is in q's second row
    (0, 3 * 8192, 8192, 4096, 9), (5 * 8192, 0, 4096, 8192, 9),     # other strides
])
def test_attend_refuses_output_rows_over_query_rows(q, out, qs, os, n):
    """Rows of 8192 bytes; strides in elements of 2 bytes."""
    kv, p = kv_struct(), attend_params(q_lens=[n], q_stride=qs, out_stride=os)
    st, need = attend_size(kv, p)
    base = FAKE + 0x1000000
    assert W.lib().wi_attend(base + q, C.byref(kv), C.byref(p), base + out, None, FAKE, need, None) == W.WI_ERR_INVALID_ARG


def test_attend_splits_only_where_blocks_are_few():
    # a prompt has blocks enough: status word only, no parts
    assert attend_size(kv_struct(seq=[65536]), attend_params())[1] == 256
    # a single token over the same cache: parts of Hq rows a run
    st, n = attend_size(kv_struct(seq=[65536]), attend_params(q_lens=[1]))
    assert st == W.WI_OK and n >= 256 + 4 * 32 * (128 + 2) * 4
    # many single tokens: their units alone fill the SMs, no longer than one another
    st, n = attend_size(kv_struct(seq=[1024] * 256), attend_params(q_lens=[1] * 256))
    assert st == W.WI_OK and n == 256


def attend_bound(batch, max_seq, max_q, dtype=W.WI_BF16, H=8, d=128, Hq=32):
    n = C.c_size_t()
    return W.lib().wi_attend_workspace_bound(dtype, batch, H, d, Hq, max_seq, max_q, C.byref(n)), n.value


def test_attend_workspace_is_not_monotone_in_the_lengths():
    """What wi_attend_workspace_bound is for: one token over 4366 keys needs more
    than over 4657, a chunk of 512 nothing at the start of its prompt."""
    size = lambda T, n: attend_size(kv_struct(seq=[T]), attend_params(q_lens=[n]))[1]  # noqa: E731
    assert size(4366, 1) > size(4657, 1) and size(512, 512) < size(2048, 512)


@pytest.mark.parametrize("dtype", [W.WI_BF16, W.WI_F32])
@pytest.mark.parametrize("H,G,d", [(8, 4, 128), (1, 1, 64), (16, 8, 128)])
@pytest.mark.parametrize("batch", [1, 16, 200])
def test_attend_workspace_bound_holds(dtype, H, G, d, batch):
    """For whole batches and parts of them, decode steps, chunks, prompts and
    mixtures, at every length up to the bound's."""
    import random
    rng = random.Random(f"{dtype} {H} {d} {batch}")
    over = dict(dtype=dtype, n_kv_heads=H, head_dim=d, page_size=1024, max_pages=1 << 20)
    seen = 256
    for _ in range(40):
        top = int(2 ** rng.uniform(0, 17))
        most = min(top, int(2 ** rng.uniform(0, 12)))
        st, bound = attend_bound(batch, top, most, dtype, H, d, H * G)
        assert st == W.WI_OK and bound % 256 == 0
        for _ in range(8):
            lens = [rng.randint(0, top) if rng.random() < 0.5 else top for _ in range(rng.randint(1, batch))]
            step = rng.choice([1, most])
            q_lens = [min(T, rng.choice([0, 1, step, most])) for T in lens]
            st, n = attend_size(kv_struct(seq=lens, **over), attend_params(H * G, q_lens=q_lens))
            assert st == W.WI_OK and n <= bound
            seen = max(seen, n)
    assert seen > 256


def test_attend_workspace_bound_grows_and_is_moderate():
    for dtype in (W.WI_BF16, W.WI_F32):
        for k, far in ((0, 256), (1, 1 << 20), (2, 4096)):
            at, last = [16, 20000, 40], 0
            for x in sorted({1, 2, 3, 5, 16, 17, 31, 32, 33, 64, 65, 100, 256, far}):
                at[k] = min(x, far)
                n = attend_bound(*at, dtype=dtype)[1]
                assert n >= last
                last = n
    assert attend_bound(1, 131072, 1)[1] < 3e6 and attend_bound(256, 1 << 20, 4096)[1] < 3.2e8
    assert attend_bound(64, 256, 256)[1] == 256      # two tiles of keys are never split


@pytest.mark.parametrize("over,expect", [
    (dict(), W.WI_OK), (dict(batch=0), W.WI_ERR_INVALID_ARG), (dict(batch=257), W.WI_ERR_UNSUPPORTED),
    (dict(dtype=7), W.WI_ERR_INVALID_ARG), (dict(H=0), W.WI_ERR_INVALID_ARG), (dict(d=96), W.WI_ERR_UNSUPPORTED),
    (dict(Hq=12), W.WI_ERR_INVALID_ARG), (dict(Hq=24), W.WI_ERR_UNSUPPORTED),
    (dict(max_seq=-1), W.WI_ERR_INVALID_ARG), (dict(max_q=-1), W.WI_ERR_INVALID_ARG),
    (dict(max_seq=0, max_q=0), W.WI_OK), (dict(max_seq=2 ** 31 - 1, max_q=2 ** 31 - 1), W.WI_OK),
])
def test_attend_workspace_bound_refusals(over, expect):
    assert attend_bound(**{**dict(batch=4, max_seq=100, max_q=10), **over})[0] == expect


def test_python_checks_name_the_argument():
    kv = W.KVCache(torch.zeros(4, 2, 16, 64), torch.zeros(4, 2, 16, 64),
                   torch.zeros(1, 4, dtype=torch.int32), [40])
    with pytest.raises(ValueError, match="q:"):
        W.attend(torch.zeros(40, 4, 64, dtype=torch.bfloat16), kv, W.AttendParams(4))
    with pytest.raises(ValueError, match="fewer rows"):
        W.attend(torch.zeros(39, 4, 64), kv, W.AttendParams(4))
    with pytest.raises(ValueError, match="must not overlap"):
        W.attend(torch.zeros(1, 4, 64).expand(40, 4, 64), kv, W.AttendParams(4))
    with pytest.raises(ValueError, match="heads of a token"):
        W.attend(torch.zeros(40, 64, 4).transpose(1, 2), kv, W.AttendParams(4))
    with pytest.raises(ValueError, match="one entry per sequence"):
        W.attend(torch.zeros(40, 4, 64), kv, W.AttendParams(4, [1, 2]))
    with pytest.raises(ValueError, match="k_pool"):      # not on a GPU
        W.attend(torch.zeros(40, 4, 64), kv, W.AttendParams(4))
    with pytest.raises(ValueError, match="k_pool"):
        W.append_kv(torch.zeros(3, 2, 64), torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32),
                    kv.k_pool, kv.v_pool)
    table = W.PageTable.empty(2, 4, 16, 8, "cpu")
    assert table.free_pages.tolist() == list(range(7, -1, -1)) and table.n_free.tolist() == [8]
    with pytest.raises(ValueError, match="block_table"):
        W.plan_pages(table, torch.ones(2, dtype=torch.int32), 8)


@pytest.mark.parametrize("capacity", [-1, 2 ** 31, 2 ** 32 + 5])
def test_plan_capacity_fits_an_int(capacity):
    """(2^32 + 5 went to the library as 5.)"""
    table = W.PageTable.empty(2, 4, 16, 8, "cpu")
    with pytest.raises(ValueError, match="capacity"):
        W.plan_pages(table, torch.ones(2, dtype=torch.int32), capacity)


def test_cache_lengths_may_change_between_calls():
    kv = W.KVCache(torch.zeros(4, 2, 16, 64), torch.zeros(4, 2, 16, 64),
                   torch.zeros(2, 4, dtype=torch.int32), [40, 3])
    prm = W.AttendParams(4)
    one = kv.c_struct()
    assert prm.n_queries(kv) == 43 and kv._struct() is kv._struct()
    kv.seq_lens[1] += 1
    assert prm.n_queries(kv) == 44
    assert [kv._struct().seq_lens[b] for b in range(2)] == [40, 4]
    assert [kv.c_struct().seq_lens[b] for b in range(2)] == [40, 4]
    kv.seq_lens.pop()
    assert kv._struct().batch == kv.c_struct().batch == 1 and prm.n_queries(kv) == 40
    assert one.batch == 2 and [one.seq_lens[b] for b in range(2)] == [40, 3]
    mine = kv.c_struct()      # a caller's own: changing it changes no later call
    mine.batch = 7
    assert kv._struct().batch == 1


def test_plain_plan_by_hand():
    # page 4; request 0 has 5 tokens (pages 9, 3) and gets 4: one new page;
    # request 1 is new and gets 5: two pages; the stack's end goes first
    got = S.plan_reference([[9, 3, -1], [-1, -1, -1]], [5, 0], [4, 5], [1, 0, 7, 2, 6], 4, 4, 10, 10)
    table, slots, positions, starts, lens, n_free = got
    assert table == [[9, 3, 2], [7, 0, -1]] and n_free == 1 and lens == [9, 5]
    assert slots == [13, 14, 15, 8, 28, 29, 30, 31, 0, -1] and starts == [0, 4, 9]
    assert positions == [5, 6, 7, 8, 0, 1, 2, 3, 4, -1]
    # three pages needed, two free: nothing happens
    got = S.plan_reference([[9, 3, -1], [-1, -1, -1]], [5, 0], [4, 5], [1, 0], 2, 4, 10, 10)
    assert got == ([[9, 3, -1], [-1, -1, -1]], [-1] * 10, [-1] * 10, [0, 0, 0], [5, 0], 2)


def test_plain_attention_by_hand():
    # one head, d = 64, two tokens on page 1; scores 0 and 8 * ln 2 / 8 = ln 2
    k, v = torch.zeros(2, 1, 2, 64), torch.zeros(2, 1, 2, 64)
    k[1, 0, 1, 0], v[1, 0, 0, 0], v[1, 0, 1, 0] = 8 * 0.6931471805599453, 3.0, 6.0
    q = torch.zeros(2, 1, 64)
    q[:, 0, 0] = 1.0
    out, lse, mag, dot = S.attend_reference(q, k, v, torch.tensor([[1]]), [2], [2])
    assert out[0, 0, 0] == 3.0 and lse[0, 0] == 0.0
    assert abs(out[1, 0, 0] - (3 + 2 * 6) / 3) < 1e-6 and abs(lse[1, 0] - 1.0986123) < 1e-6
