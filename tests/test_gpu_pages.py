"""The paged-cache calls on cuda:0 through the C ABI against the fp64 oracle:
types, head layouts, page sizes, lengths from none to long ones, strides, bad
pages, stale rows, streams, captured graphs, and a run of them together on
pages that kvtc_decode restored."""
import numpy as np
import pytest
import torch

import kv_cache_transform_amd as K
import oracle.kvtc_pages as OP
import synth
from gpu_util import DEV, DevCodec, oracle_artifact, to_dev_bytes

pytestmark = pytest.mark.gpu

BF16, F32 = K.KVTC_BF16, K.KVTC_F32
TORCH = {BF16: torch.bfloat16, F32: torch.float32}
NAN = float("nan")


def dev(x, dtype=torch.int32):
    return torch.tensor(np.array(x), dtype=dtype).to(DEV)


def f64(t):
    return t.detach().double().cpu().numpy()


def case(seed, dtype, heads, group, dim, bs, lens, spare=3, extra=1, stale=NAN, gain=1.0):
    """A paged cache with the given lengths: rows behind a request's last token and pages that no request has
    hold `stale`, table entries behind a request's pages a page far outside."""
    r = np.random.default_rng(seed)
    need = [OP.n_pages(max(n, 0), bs) for n in lens]
    n_blocks = sum(need) + spare
    width = max(need + [1])
    stride = width + extra
    order = r.permutation(n_blocks)
    table = np.full((len(lens), stride), 2**31 - 1, np.int64)
    live = np.zeros((n_blocks, bs), bool)
    at = 0
    for i, n in enumerate(lens):
        table[i, :need[i]] = order[at:at + need[i]]
        at += need[i]
        for j in range(need[i]):
            live[table[i, j], :min(bs, n - j * bs)] = True
    shape = (n_blocks, bs, heads, dim)
    k = r.normal(size=shape) * np.where(np.arange(dim) % 17 == 3, 4.0, 1.0) + 0.3
    v = r.normal(size=shape) + 0.1
    q = r.normal(size=(len(lens), heads * group, dim)) * gain
    if stale is not None:
        k[~live] = stale
        v[~live] = stale
    put = lambda a: torch.from_numpy(a.astype(np.float32)).to(DEV).to(TORCH[dtype]).contiguous()  # noqa: E731
    c = dict(dtype=dtype, heads=heads, group=group, dim=dim, bs=bs, lens=np.array(lens), width=width, stride=stride,
             n_blocks=n_blocks, live=live, table=table, k=put(k), v=put(v), q=put(q))
    c["dtable"], c["dlens"] = dev(table), dev(lens)
    c["status"] = torch.zeros(len(lens), dtype=torch.int32, device=DEV)
    c["pages"] = K.make_pages(c["k"], c["v"], n_blocks, bs, heads, dim, dtype)
    c["req"] = K.make_requests(c["dtable"], width, c["dlens"], len(lens), status=c["status"], table_stride=stride)
    return c


def attend(c, scale, blocks=None, q=None, out=None, lse=None, stream=None, **strides):
    """-> (out, lse, status) after one call; blocks: device int32 [n, heads, budget]."""
    n, hq = len(c["lens"]), c["heads"] * c["group"]
    q = c["q"] if q is None else q
    out = torch.full((n, hq * c["dim"]), 7.0, dtype=TORCH[c["dtype"]], device=DEV) if out is None else out
    lse = torch.full((n, hq), 7.0, dtype=torch.float32, device=DEV) if lse is None else lse
    queries = K.make_queries(q, out, hq, scale, lse=lse, **strides)
    sel = None if blocks is None else K.make_selection(blocks, blocks.shape[-1])
    ws = torch.full((K.kvtc_page_workspace_bytes(c["pages"], c["req"], queries, sel),), 0xFF, dtype=torch.uint8, device=DEV)
    K.kvtc_page_attend(c["pages"], c["req"], queries, sel, ws, stream=stream or torch.cuda.current_stream())
    torch.cuda.synchronize()
    return out, lse, c["status"].cpu().numpy()


def check_attend(c, scale, out, lse, blocks=None, status=None):
    """Against the oracle. A score is off by at most (D + 4) 2^-24 of scale * sum |q k| (fp32 products and sums,
    the scaling and the base change of the exponential), a weight by that, the exponential's own 2^-22 and, for bf16
    pages, 2^-15 (two bf16 terms); sums over n tokens by n / 8 + 64 additions' 2^-24; out once more by its rounding."""
    want, wlse, wst, slack = OP.attend(f64(c["q"]), f64(c["k"]), f64(c["v"]), c["table"], c["lens"], c["width"], scale, blocks)
    got, glse = f64(out).reshape(want.shape), f64(lse)
    eps = torch.finfo(TORCH[c["dtype"]]).eps / 2
    for i in range(want.shape[0]):
        for x in range(want.shape[1]):
            big, mass, n = slack[i][x]
            if n == 0:
                assert np.all(got[i, x] == 0) and glse[i, x] == -np.inf, (i, x)
                continue
            ds = (c["dim"] + 4) * 2.0**-24 * (big + abs(wlse[i, x])) + 2.0**-22
            rel = 2 * ds + (n / 8 + 64) * 2.0**-24 + (2.0**-15 if c["dtype"] == BF16 else 0.0)
            tol = eps * np.abs(want[i, x]) + rel * (mass + np.abs(want[i, x])) * (1 + eps) + 1e-30
            err = np.abs(got[i, x] - want[i, x])
            assert np.all(err <= tol), (i, x, n, float((err / tol).max()))
            assert abs(glse[i, x] - wlse[i, x]) <= rel + 2.0**-23 * abs(wlse[i, x]), (i, x, glse[i, x], wlse[i, x])
    if status is not None:
        assert np.array_equal(status, wst), (status, wst)


# ------------------------------------------------------------------- attention ---

LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300, 511, 1000]

ATTEND = [
    # dtype, heads, group, dim, page, lengths
    (BF16, 8, 4, 128, 16, LENS), (F32, 8, 4, 128, 16, LENS), (BF16, 2, 7, 128, 16, [700, 3, 1024]),
    (BF16, 3, 4, 64, 16, LENS), (F32, 3, 4, 64, 16, LENS), (BF16, 1, 1, 64, 16, [1]), (F32, 1, 1, 8, 1, [1, 0, 5]),
    (BF16, 2, 1, 8, 1, [40, 1, 9]), (BF16, 2, 3, 16, 3, [100, 2, 7]), (BF16, 2, 16, 80, 20, [333, 20, 19, 21]),
    (F32, 2, 16, 80, 20, [333, 20, 19, 21]), (BF16, 1, 17, 96, 8, [130, 8, 4]), (F32, 1, 17, 96, 8, [130, 8, 4]),
    (BF16, 1, 40, 128, 64, [500, 64, 1]), (BF16, 2, 8, 192, 32, [257, 31]), (F32, 2, 8, 192, 32, [257, 31]),
    (BF16, 2, 5, 256, 16, [400, 17]), (F32, 2, 5, 256, 16, [400, 17]), (BF16, 2, 2, 200, 24, [100, 25]),
    # pages that cut the kernels' groups of 8 or 4 positions, and pages smaller than a group
    (BF16, 2, 4, 128, 9, [1, 8, 9, 10, 17, 18, 19, 300, 0]), (BF16, 1, 4, 64, 11, [260, 11, 10, 12, 1]), (BF16, 2, 3, 256, 12, [130, 13, 12]),
    (BF16, 2, 16, 128, 15, [600, 14, 15, 16]), (F32, 2, 3, 128, 5, [200, 4, 5, 6, 1]), (F32, 1, 2, 256, 6, [90, 7, 0]),
    (F32, 3, 4, 64, 9, [300, 8, 9, 10]), (BF16, 2, 4, 128, 7, [300, 6, 7, 8]), (F32, 2, 4, 64, 3, [100, 2, 3, 4]), (F32, 2, 4, 128, 2, [70]),
    (BF16, 1, 4, 128, 100, [1, 99, 100, 101, 950]), (BF16, 4, 2, 40, 5, [77, 4, 5, 6]), (F32, 4, 2, 24, 7, [77, 6, 7, 8]),
]


@pytest.mark.parametrize("i", range(len(ATTEND)))
def test_attend(i):
    dtype, heads, group, dim, bs, lens = ATTEND[i]
    c = case(i, dtype, heads, group, dim, bs, lens)
    print(f"attend {ATTEND[i]}", flush=True)
    out, lse, st = attend(c, dim ** -0.5)
    check_attend(c, dim ** -0.5, out, lse, status=st)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens", [[9000], [5000, 1, 0, 3], [40, 6000, 40, 2500, 1], [300] * 37, [129, 128, 1] * 30, [20000]])
def test_attend_long_lengths_are_split_and_joined(dtype, lens):
    c = case(5, dtype, 2, 4, 64, 16, lens)
    out, lse, st = attend(c, 0.125)
    check_attend(c, 0.125, out, lse, status=st)


@pytest.mark.parametrize("n", [700, 4096])
def test_attend_many_requests(n):
    r = np.random.default_rng(8)
    lens = [int(x) for x in r.integers(0, 90, n)]
    c = case(9, BF16, 1, 2, 64, 16, lens)
    out, lse, st = attend(c, 0.125)
    check_attend(c, 0.125, out, lse, status=st)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale,gain", [(0.0, 1.0), (-0.2, 1.0), (1.0, 1.0), (0.125, 60.0), (1e-4, 1.0)])
def test_attend_scales(dtype, scale, gain):
    c = case(11, dtype, 2, 4, 64, 16, [1, 40, 333], gain=gain)
    out, lse, st = attend(c, scale)
    check_attend(c, scale, out, lse, status=st)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bs", [16, 12, 9, 6, 3])
@pytest.mark.parametrize("stale", [NAN, float("inf"), float("-inf"), 3.0e38])
def test_attend_never_uses_stale_rows(dtype, bs, stale):
    c = case(12, dtype, 2, 4, 128, bs, [1, 15, 17, 100, 0], stale=stale)
    out, lse, st = attend(c, 0.1)
    check_attend(c, 0.1, out, lse, status=st)


def test_attend_writes_where_it_reads():
    """out may take the place of q: a row's queries are read before any of its results are written."""
    c = case(50, BF16, 2, 4, 64, 16, [3000, 1, 40, 0])
    ref, lse, _ = attend(c, 0.125)
    buf = c["q"].reshape(4, 512).clone()
    out, lse2, _ = attend(c, 0.125, q=buf, out=buf)
    assert torch.equal(out, ref) and torch.equal(lse, lse2)


def test_attend_requests_that_share_pages():
    c = case(51, F32, 2, 2, 64, 16, [200, 100, 64])
    c["table"][1, :7] = c["table"][0, :7]
    c["table"][2, :3] = c["table"][0, 2:5]
    c["dtable"].copy_(dev(c["table"]))
    out, lse, st = attend(c, 0.125)
    check_attend(c, 0.125, out, lse, status=st)


def test_attend_strided_rows_and_what_lies_beside_them():
    c = case(13, BF16, 2, 4, 64, 16, [50, 0, 200])
    wide = torch.full((3, 3 * 512 + 8), 5.0, dtype=torch.bfloat16, device=DEV)
    wide[:, 512:1024] = c["q"].reshape(3, -1)
    out = torch.full((3, 1024), 7.0, dtype=torch.bfloat16, device=DEV)
    o, lse, st = attend(c, 0.125, q=wide[:, 512:], out=out[:, 256:], q_stride=wide.stride(0), out_stride=1024)
    check_attend(c, 0.125, out[:, 256:768], lse, status=st)
    assert bool((out[:, :256] == 7).all()) and bool((out[:, 768:] == 7).all())


def test_attend_without_lse_and_status():
    c = case(14, BF16, 2, 4, 64, 16, [50, 300])
    ref, _, _ = attend(c, 0.125)
    out = torch.empty_like(ref)
    queries = K.make_queries(c["q"], out, 8, 0.125)
    req = K.make_requests(c["dtable"], c["width"], c["dlens"], 2, table_stride=c["stride"])
    ws = torch.empty(K.kvtc_page_workspace_bytes(c["pages"], req, queries), dtype=torch.uint8, device=DEV)
    K.kvtc_page_attend(c["pages"], req, queries, None, ws, stream=torch.cuda.current_stream())
    assert torch.equal(out, ref)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bs", [16, 13, 5])
def test_attend_leaves_out_bad_pages_and_lengths(dtype, bs):
    c = case(15, dtype, 2, 4, 64, bs, [40, 100, 64, 10, 33])
    c["table"][1, 2], c["table"][2, 0], c["table"][2, 3], c["table"][3, 0] = -1, c["n_blocks"], -2**31, 2**31 - 1
    c["dtable"].copy_(dev(c["table"]))
    c["lens"] = np.array([40, 100, 64, 10, c["width"] * bs + 1])
    c["dlens"].copy_(dev(c["lens"]))
    out, lse, st = attend(c, 0.125)
    check_attend(c, 0.125, out, lse, status=st)
    assert list(st) == [0, -1, -1, -1, -1]
    c["lens"][4], c["status"][:] = -5, 0
    c["dlens"].copy_(dev(c["lens"]))
    out, lse, st = attend(c, 0.125)
    check_attend(c, 0.125, out, lse, status=st)
    # a status word that holds an error is not cleared
    c["status"][0] = -3
    assert list(attend(c, 0.125)[2]) == [-3, -1, -1, -1, -1]


@pytest.mark.parametrize("dtype,heads,group,dim,bs", [(BF16, 2, 4, 128, 16), (F32, 2, 4, 64, 16), (BF16, 3, 5, 80, 5), (BF16, 1, 20, 64, 32),
                                                       (BF16, 2, 4, 128, 12), (F32, 1, 4, 64, 6), (BF16, 2, 4, 64, 9), (F32, 2, 2, 128, 3)])
def test_attend_over_selected_pages(dtype, heads, group, dim, bs):
    lens = [0, 1, bs, 5 * bs - 1, 40 * bs + 1]
    c = case(16, dtype, heads, group, dim, bs, lens)
    r = np.random.default_rng(3)
    blocks = np.full((len(lens), heads, 9), -1, np.int64)
    for i, n in enumerate(lens):
        for h in range(heads):
            m = OP.n_pages(n, bs)
            some = r.permutation(m)[:r.integers(0, min(m, 9) + 1)]
            blocks[i, h, :len(some)] = np.sort(some) if i % 2 else some
    blocks[1, 0, :3] = [5, -7, 2**31 - 1]         # past the request's pages: left out
    blocks[4, 0, 0], blocks[4, 0, 5] = -1, 40      # a gap, and the last, partly filled page
    out, lse, st = attend(c, 0.2, blocks=dev(blocks))
    check_attend(c, 0.2, out, lse, blocks=blocks, status=st)


def test_attend_with_a_large_budget_is_split_too():
    c = case(17, BF16, 2, 4, 128, 16, [9000, 300])
    blocks = np.full((2, 2, 520), -1, np.int64)
    r = np.random.default_rng(4)
    for i in range(2):
        for h in range(2):
            m = min(520, OP.n_pages(int(c["lens"][i]), 16))
            blocks[i, h, :m] = np.sort(r.permutation(OP.n_pages(int(c["lens"][i]), 16))[:m])
    out, lse, st = attend(c, 0.2, blocks=dev(blocks))
    check_attend(c, 0.2, out, lse, blocks=blocks, status=st)
    every = np.full((2, 2, 563), -1, np.int64)
    for i in range(2):
        m = OP.n_pages(int(c["lens"][i]), 16)
        every[i, :, :m] = np.arange(m)
    out, lse, st = attend(c, 0.2, blocks=dev(every))
    check_attend(c, 0.2, out, lse, status=st)


def test_attend_equal_calls_give_equal_bits():
    c = case(18, BF16, 4, 4, 128, 16, [7000, 12, 900, 0])
    a, la, _ = attend(c, 0.1)
    for _ in range(5):
        b, lb, _ = attend(c, 0.1)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_attend_pages_past_2_31_elements():
    heads, dim, bs = 8, 128, 16
    n_blocks = (1 << 31) // (bs * heads * dim) + 40          # over 2^31 elements of K, and of V
    k = torch.empty((n_blocks, bs, heads, dim), dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    small = case(19, BF16, heads, 4, dim, bs, [500, 33])
    far = np.array(small["table"])
    for i in range(2):
        for j in range(OP.n_pages(int(small["lens"][i]), bs)):
            far[i, j] = n_blocks - 1 - small["table"][i, j]
            k[int(far[i, j])] = small["k"][int(small["table"][i, j])]
            v[int(far[i, j])] = small["v"][int(small["table"][i, j])]
    a, la, _ = attend(small, 0.1)
    big = dict(small, k=k, v=v, dtable=dev(far), pages=K.make_pages(k, v, n_blocks, bs, heads, dim, BF16))
    big["req"] = K.make_requests(big["dtable"], big["width"], big["dlens"], 2, status=big["status"], table_stride=big["stride"])
    b, lb, st = attend(big, 0.1)
    assert torch.equal(a, b) and torch.equal(la, lb) and not st.any()
    # written there as well
    rows = torch.randn(4, 1024, device=DEV).bfloat16()
    slots = dev([n_blocks * bs - 1, 2**21 + 5, 3, -1])
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    K.kvtc_page_write(big["pages"], K.make_page_rows(rows, rows, 4, slots, BF16, 1024, 1024, status=word), torch.cuda.current_stream())
    flat = k.view(-1, 1024)
    for i, s in enumerate([n_blocks * bs - 1, 2**21 + 5, 3]):
        assert torch.equal(flat[s], rows[i])
    assert int(word) == 0
    bnd = torch.empty((n_blocks, 2, 1024), dtype=torch.bfloat16, device=DEV)
    K.kvtc_page_bounds(big["pages"], big["req"], None, bnd, stream=torch.cuda.current_stream())
    p = int(far[0, 0])
    assert torch.equal(bnd[p, 1], k[p].view(bs, 1024).amax(0)) and torch.equal(bnd[p, 0], k[p].view(bs, 1024).amin(0))


# ------------------------------------------------------ block tables, slot maps ---

def run_tables(old, new, bs, free, n_blocks, table, width, n_slots, free_from=None, pad=2):
    stride = table.shape[1]
    d = dict(old=None if old is None else dev(old), new=dev(new), free=dev(free), table=dev(table),
             slots=torch.full((n_slots + pad,), 77, dtype=torch.int32, device=DEV),
             starts=torch.full((len(new) + 1,), 77, dtype=torch.int32, device=DEV),
             taken=torch.full((1,), 77, dtype=torch.int32, device=DEV), status=torch.zeros(len(new), dtype=torch.int32, device=DEV),
             ff=None if free_from is None else dev([free_from]))
    plan = K.make_page_plan(d["old"], d["new"], len(new), bs, d["free"], len(free), n_blocks, d["table"], width, d["slots"], n_slots,
                            free_from=d["ff"], starts=d["starts"], taken=d["taken"], status=d["status"], table_stride=stride)
    K.kvtc_page_tables(plan, torch.cuda.current_stream())
    torch.cuda.synchronize()
    want = OP.tables(np.zeros(len(new), int) if old is None else old, new, bs, free, free_from or 0, n_blocks, table, width, n_slots)
    got = [d[x].cpu().numpy() for x in ("table", "slots", "starts", "taken", "status")]
    assert np.array_equal(got[0], want[0])
    assert np.array_equal(got[1][:n_slots], want[1]) and np.all(got[1][n_slots:] == 77)
    assert np.array_equal(got[2], want[2]) and got[3][0] == want[3] and np.array_equal(got[4], want[4]), (got[4], want[4])
    return want


def tables_case(seed, n, bs, longest, grow, extra=2):
    r = np.random.default_rng(seed)
    old = r.integers(0, longest + 1, n)
    new = old + (r.integers(0, grow + 1, n) if grow else 0)
    width = max(1, OP.n_pages(int(new.max()), bs))
    table = np.full((n, width + extra), -9, np.int64)
    need = [OP.n_pages(int(x), bs) for x in old]
    total = sum(OP.n_pages(int(x), bs) for x in new) + 6
    ids = r.permutation(total)
    at = 0
    for i in range(n):
        table[i, :need[i]] = ids[at:at + need[i]]
        at += need[i]
    return old, new, table, width, ids[at:], total


@pytest.mark.parametrize("n,bs,longest,grow", [(1, 16, 0, 1), (1, 16, 31, 1), (3, 1, 5, 4), (64, 16, 500, 1), (300, 16, 90, 40), (257, 24, 100, 0),
                                               (5, 7, 1000, 5000), (4096, 16, 30, 3), (256, 64, 10, 700)])
def test_tables(n, bs, longest, grow):
    old, new, table, width, free, total = tables_case(n + bs, n, bs, longest, grow)
    tokens = int((new - old).sum())
    run_tables(old, new, bs, free, total, table, width, tokens)
    run_tables(old, new, bs, free, total, table, width, tokens + 1500)
    # from the middle of the pool, too few pages, too few slots, no pool at all
    run_tables(old, new, bs, np.concatenate([[0, 0, 0], free]), total, table, width, tokens, free_from=3)
    run_tables(old, new, bs, free[:max(0, (len(free) - 6) // 2)], total, table, width, tokens)
    run_tables(old, new, bs, free, total, table, width, tokens // 2)
    run_tables(old, new, bs, free[:0], total, table, width, tokens)
    run_tables(old, new, bs, free, total, table, width, 0)


def test_tables_from_nothing_and_bad_requests():
    new = np.array([0, 33, 16, 1, 70])
    table = np.full((5, 6), -9, np.int64)
    run_tables(None, new, 16, np.arange(20)[::-1], 20, table, 5, 130)
    old = np.array([0, -1, 20, 5, 2**31 - 1])
    new = np.array([81, 5, 19, 9, 2**31 - 1])       # past the table, negative, shrinking, fine, past the table
    table[3, 0] = 7
    want = run_tables(old, new, 16, np.arange(20), 20, table, 5, 130)
    assert list(want[4]) == [-1, -1, -1, 0, -1]
    # pages outside the cache, one held and one from the pool; a negative and a far free_from
    table[3, 0] = 20
    run_tables([0, 0, 0, 5, 0], [16, 16, 16, 9, 17], 16, [3, -4, 5, 6, 25], 20, table, 5, 130)
    run_tables([0, 0, 0, 5, 0], [16, 16, 16, 9, 17], 16, [3, 4, 5, 6, 7], 20, table, 5, 130, free_from=-3)
    run_tables([0, 0, 0, 5, 0], [16, 16, 16, 9, 17], 16, [3, 4, 5, 6, 7], 20, table, 5, 130, free_from=2**31 - 1)


def test_tables_without_the_optional_outputs():
    new, table = dev([5, 40]), torch.full((2, 3), -1, dtype=torch.int32, device=DEV)
    slots = torch.empty(45, dtype=torch.int32, device=DEV)
    K.kvtc_page_tables(K.make_page_plan(None, new, 2, 16, dev([4, 2, 0, 1]), 4, 5, table, 3, slots, 45), torch.cuda.current_stream())
    assert table.tolist() == [[4, -1, -1], [2, 0, 1]]
    assert slots.tolist() == list(range(64, 69)) + list(range(32, 48)) + list(range(16)) + list(range(16, 24))


# ------------------------------------------------------------------------ write ---

@pytest.mark.parametrize("heads,dim,bs,n", [(8, 128, 16, 70), (3, 64, 16, 1), (1, 8, 1, 9), (2, 40, 5, 333), (5, 200, 24, 64), (1, 256, 16, 3000)])
@pytest.mark.parametrize("src", [BF16, F32])
@pytest.mark.parametrize("dst", [BF16, F32])
def test_write(heads, dim, bs, n, src, dst):
    F = heads * dim
    n_blocks = OP.n_pages(n, bs) + 2
    g = torch.Generator(device=DEV)
    g.manual_seed(n)
    k = torch.full((n_blocks * bs, F), 7.0, dtype=TORCH[dst], device=DEV)
    v = torch.full_like(k, 8.0)
    slots = torch.randperm(n_blocks * bs, generator=g, device=DEV)[:n].to(torch.int32)
    slots[n // 3::5] = -1
    for width, off in ((4 * F, 2 * F), (F + 1, 1), (F, 0), (4 * F + 3, 2 * F)):      # slices, odd strides and offsets, dense
        wide = torch.randn(n, width + F, generator=g, device=DEV).to(TORCH[src])
        wide[0, :3] = torch.tensor([NAN, float("inf"), -0.0])
        rows_k, rows_v = wide[:, off:off + F], wide[:, width:]
        word = torch.zeros(1, dtype=torch.int32, device=DEV)
        pages = K.make_pages(k, v, n_blocks, bs, heads, dim, dst)
        K.kvtc_page_write(pages, K.make_page_rows(rows_k, rows_v, n, slots, src, wide.stride(0), wide.stride(0), status=word), torch.cuda.current_stream())
        keep = slots >= 0
        wk, wv = torch.full_like(k, 7.0), torch.full_like(v, 8.0)
        wk[slots[keep].long()], wv[slots[keep].long()] = rows_k[keep].to(TORCH[dst]), rows_v[keep].to(TORCH[dst])
        bits = torch.int16 if dst == BF16 else torch.int32
        nan = torch.isnan(wk)
        assert torch.equal(torch.isnan(k), nan) and torch.equal(k.view(bits)[~nan], wk.view(bits)[~nan])
        nan = torch.isnan(wv)
        assert torch.equal(torch.isnan(v), nan) and torch.equal(v.view(bits)[~nan], wv.view(bits)[~nan])
        assert int(word) == 0


def test_write_rounds_to_nearest_even():
    bits = np.arange(0x3F800000, 0x3F800000 + 8 * 0x2001, 0x2001, dtype=np.int64)[:8]
    edge = np.array([0x3F808000, 0x3F818000, 0x3F807FFF, 0x3F808001, 0x7F7FFFFF, 0x00008000, 0x80018000 - 2**32, 0x7F800000])
    x = torch.from_numpy(np.stack([bits, edge]).astype(np.int32)).view(torch.float32).to(DEV)
    k = torch.zeros(4, 8, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    K.kvtc_page_write(K.make_pages(k, v, 4, 1, 1, 8, BF16), K.make_page_rows(x, x, 2, dev([2, 0]), F32, 8, 8), torch.cuda.current_stream())
    assert torch.equal(k[2].view(torch.int16), x[0].bfloat16().view(torch.int16))
    assert torch.equal(v[0].view(torch.int16), x[1].bfloat16().view(torch.int16))


def test_write_slots_outside():
    k = torch.zeros(6, 64, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    x = torch.randn(5, 64, device=DEV).bfloat16()
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    K.kvtc_page_write(K.make_pages(k, v, 2, 3, 1, 64, BF16), K.make_page_rows(x, x, 5, dev([5, -1, -2**31, 0, 4]), BF16, 64, 64, status=word), torch.cuda.current_stream())
    assert int(word) == 0
    K.kvtc_page_write(K.make_pages(k, v, 2, 3, 1, 64, BF16), K.make_page_rows(x, x, 5, dev([6, 2**31 - 1, -1, -1, 1]), BF16, 64, 64, status=word), torch.cuda.current_stream())
    assert int(word) == K.KVTC_E_INVALID
    for row, i in ((5, 0), (0, 3), (4, 4), (1, 4)):
        assert torch.equal(k[row], x[i]) and torch.equal(v[row], x[i])
    assert not bool(k[2:4].any())


# ----------------------------------------------------------------------- bounds ---

@pytest.mark.parametrize("dtype,heads,dim,bs,lens", [
    (BF16, 8, 128, 16, LENS), (F32, 3, 64, 16, LENS), (BF16, 1, 8, 1, [0, 1, 9]), (F32, 2, 40, 5, [33, 4, 5, 6]), (BF16, 2, 200, 24, [100, 24, 1]),
    (BF16, 1, 64, 100, [250, 7]), (BF16, 5, 256, 32, [95, 0, 64])])
@pytest.mark.parametrize("back", [None, 0, 1, 40])
def test_bounds(dtype, heads, dim, bs, lens, back):
    c = case(21, dtype, heads, 1, dim, bs, lens)
    F = heads * dim
    since = None if back is None else np.array(lens) - back       # negative ones count as 0
    bnd = torch.full((c["n_blocks"], 2, F), 9.0, dtype=TORCH[dtype], device=DEV)
    K.kvtc_page_bounds(c["pages"], c["req"], None if since is None else dev(since), bnd, stream=torch.cuda.current_stream())
    want = np.full((c["n_blocks"], 2, F), 9.0)
    found, st = OP.bounds(f64(c["k"]), c["table"], c["lens"], c["width"], since)
    for page, (lo, hi) in found.items():
        want[page, 0], want[page, 1] = lo, hi
    assert np.array_equal(f64(bnd), want)
    assert np.array_equal(c["status"].cpu().numpy(), st)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bounds_of_special_values_and_bad_pages(dtype):
    c = case(22, dtype, 2, 1, 64, 16, [40, 100, 64, 10])
    for page, row, f, x in ((0, 3, 5, NAN), (1, 0, 6, NAN), (2, 1, 7, float("inf")), (3, 0, 8, float("-inf"))):
        i, j = divmod(page, 2)
        c["k"][int(c["table"][i, j]), row].view(-1)[f] = x
    c["table"][1, 3], c["table"][2, 2] = -1, c["n_blocks"]
    c["dtable"].copy_(dev(c["table"]))
    c["lens"] = np.array([40, 100, 64, -1])
    c["dlens"].copy_(dev(c["lens"]))
    bnd = torch.full((c["n_blocks"], 2, 128), 9.0, dtype=TORCH[dtype], device=DEV)
    K.kvtc_page_bounds(c["pages"], c["req"], None, bnd, stream=torch.cuda.current_stream())
    want = np.full((c["n_blocks"], 2, 128), 9.0)
    found, st = OP.bounds(f64(c["k"]), c["table"], c["lens"], c["width"])
    for page, (lo, hi) in found.items():
        want[page, 0], want[page, 1] = lo, hi
    assert np.array_equal(f64(bnd), want, equal_nan=True)
    assert list(c["status"].cpu().numpy()) == list(st) == [0, -1, -1, -1]


# -------------------------------------------------------------------- selection ---

def page_bounds(c):
    bnd = torch.full((c["n_blocks"], 2, c["heads"], c["dim"]), NAN, dtype=TORCH[c["dtype"]], device=DEV)
    K.kvtc_page_bounds(c["pages"], c["req"], None, bnd, stream=torch.cuda.current_stream())
    return bnd


def select(c, bnd, budget, first, last, stream=None):
    n, hq = len(c["lens"]), c["heads"] * c["group"]
    blocks = torch.full((n, c["heads"], budget), 77, dtype=torch.int32, device=DEV)
    queries, sel = K.make_queries(c["q"], None, hq, 1.0), K.make_selection(blocks, budget, first, last)
    ws = torch.full((K.kvtc_page_workspace_bytes(c["pages"], c["req"], queries, sel),), 0xFF, dtype=torch.uint8, device=DEV)
    K.kvtc_page_select(c["pages"], c["req"], queries, bnd, sel, ws, stream=stream or torch.cuda.current_stream())
    torch.cuda.synchronize()
    return blocks


def check_select(c, bnd, budget, first, last):
    got = select(c, bnd, budget, first, last).cpu().numpy()
    want, st = OP.select(f64(c["q"]), f64(bnd), c["table"], c["lens"], c["bs"], c["n_blocks"], c["width"], c["heads"], budget, first, last)
    assert np.array_equal(got, want)
    assert np.array_equal(c["status"].cpu().numpy(), st)


@pytest.mark.parametrize("dtype,heads,group,dim,bs,lens", [
    (BF16, 8, 4, 128, 16, [0, 1, 16, 17, 400, 3000]), (F32, 3, 4, 64, 16, [900, 1, 0, 33]), (BF16, 1, 1, 8, 1, [300, 7, 1]),
    (BF16, 2, 7, 80, 5, [700, 4, 5, 6]), (F32, 1, 20, 256, 24, [1000, 25]), (BF16, 2, 16, 200, 64, [4000])])
@pytest.mark.parametrize("budget,first,last", [(1, 0, 0), (3, 1, 2), (8, 2, 3), (64, 0, 1), (300, 4, 4)])
def test_select(dtype, heads, group, dim, bs, lens, budget, first, last):
    c = case(31, dtype, heads, group, dim, bs, lens)
    check_select(c, page_bounds(c), budget, first, last)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_select_many_pages(dtype):
    c = case(32, dtype, 1, 2, 16, 1, [20000, 3, 9000])
    check_select(c, page_bounds(c), 700, 3, 5)


def test_select_ties_go_to_the_lowest_index():
    c = case(33, BF16, 2, 2, 64, 16, [600, 160])
    bnd = torch.zeros((c["n_blocks"], 2, 2, 64), dtype=torch.bfloat16, device=DEV)      # every score is 0
    check_select(c, bnd, 7, 1, 2)
    bnd.copy_(torch.randint(0, 2, (c["n_blocks"], 2, 2, 1), device=DEV).bfloat16().expand_as(bnd))   # two values of a score
    c["q"].fill_(0.5)
    for budget in (1, 5, 12, 20, 37, 38, 39):
        check_select(c, bnd, budget, 0, 1)
    bnd.fill_(-0.0)
    c["q"].fill_(-0.0)
    check_select(c, bnd, 7, 0, 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_select_special_scores(dtype):
    c = case(34, dtype, 2, 2, 64, 16, [600, 160, 320])
    bnd = page_bounds(c)
    for j, x in ((3, NAN), (5, float("inf")), (7, float("-inf")), (9, NAN)):
        bnd[int(c["table"][0, j]), :, 0, 11] = x
    for budget in (1, 2, 3, 4, 6, 37, 38):
        check_select(c, bnd, budget, 0, 1)
    c["q"][1, 1, 4] = NAN              # every score of head 0 is NaN: the first ones
    c["q"][2, 2, 4] = float("inf")
    check_select(c, bnd, 4, 1, 1)


def test_select_skips_bad_pages_and_lengths():
    c = case(35, BF16, 2, 2, 64, 16, [600, 160, 100])
    bnd = page_bounds(c)
    c["table"][0, 0], c["table"][0, 20], c["table"][1, 9] = -1, c["n_blocks"], 2**31 - 1
    c["dtable"].copy_(dev(c["table"]))
    c["lens"] = np.array([600, 160, c["width"] * 16 + 1])
    c["dlens"].copy_(dev(c["lens"]))
    check_select(c, bnd, 8, 1, 2)
    c["status"].zero_()
    check_select(c, bnd, 60, 1, 2)


def test_the_score_bounds_the_products():
    c = case(36, BF16, 2, 4, 64, 16, [500])
    bnd, q, k = f64(page_bounds(c)), f64(c["q"]), f64(c["k"])
    for h in range(2):
        for j in range(OP.n_pages(500, 16)):
            page, rows = int(c["table"][0, j]), min(16, 500 - 16 * j)
            best = (k[page, :rows, h] @ q[0, 4 * h:4 * h + 4].T).max(0).sum()
            assert OP.scores(q[0, 4 * h:4 * h + 4], bnd[page, 0, h], bnd[page, 1, h]) >= best * (1 - 2.0**-23) - 1e-6


# -------------------------------------------------------------- used in earnest ---

def test_select_and_attend_share_a_workspace():
    c = case(41, BF16, 2, 4, 128, 16, [5000, 40, 0, 900])
    bnd = page_bounds(c)
    blocks = torch.empty((4, 2, 24), dtype=torch.int32, device=DEV)
    out, lse = torch.empty((4, 1024), dtype=torch.bfloat16, device=DEV), torch.empty((4, 8), device=DEV)
    queries, sel = K.make_queries(c["q"], out, 8, 0.1, lse=lse), K.make_selection(blocks, 24, 1, 2)
    ws = torch.empty(K.kvtc_page_workspace_bytes(c["pages"], c["req"], queries, sel), dtype=torch.uint8, device=DEV)
    s = torch.cuda.current_stream()
    for _ in range(3):
        K.kvtc_page_select(c["pages"], c["req"], queries, bnd, sel, ws, stream=s)
        K.kvtc_page_attend(c["pages"], c["req"], queries, sel, ws, stream=s)
    torch.cuda.synchronize()
    check_attend(c, 0.1, out, lse, blocks=blocks.cpu().numpy(), status=c["status"].cpu().numpy())


def test_two_streams_at_once():
    cs = [case(42 + i, BF16, 2, 4, 128, 16, [6000, 40 + i, 0]) for i in range(2)]
    alone = [attend(c, 0.1)[:2] for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    outs, keep = [], []
    for c, s in zip(cs, streams):
        out, lse = torch.empty((3, 1024), dtype=torch.bfloat16, device=DEV), torch.empty((3, 8), device=DEV)
        queries = K.make_queries(c["q"], out, 8, 0.1, lse=lse)
        ws = torch.empty(K.kvtc_page_workspace_bytes(c["pages"], c["req"], queries), dtype=torch.uint8, device=DEV)
        outs.append((out, lse))
        keep.append((queries, ws))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, (queries, ws) in zip(cs, streams, keep):
            K.kvtc_page_attend(c["pages"], c["req"], queries, None, ws, stream=s)
    torch.cuda.synchronize()
    for (a, la), (b, lb) in zip(alone, outs):
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_two_graphs_share_a_workspace():
    """Two captured batches of different sizes on one workspace, replayed in turn with eager work between."""
    cs = [case(60, BF16, 2, 4, 128, 16, [4000, 3, 0, 700]), case(61, BF16, 1, 7, 64, 20, [90, 2500])]
    want, outs, calls = [], [], []
    for c in cs:
        n, hq = len(c["lens"]), c["heads"] * c["group"]
        want.append(attend(c, 0.1)[:2])
        out = torch.zeros((n, hq * c["dim"]), dtype=torch.bfloat16, device=DEV)
        lse = torch.zeros((n, hq), device=DEV)
        outs.append((out, lse))
        calls.append((c, K.make_queries(c["q"], out, hq, 0.1, lse=lse)))
    ws = torch.full((max(K.kvtc_page_workspace_bytes(c["pages"], c["req"], q) for c, q in calls),), 0xA5, dtype=torch.uint8, device=DEV)
    graphs = []
    side = torch.cuda.Stream()
    for c, q in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            K.kvtc_page_attend(c["pages"], c["req"], q, None, ws, stream=side)
        graphs.append(g)
    for i in (0, 1, 0, 0, 1, 1, 0):
        for x in outs[i]:
            x.zero_()
        graphs[i].replay()
        if i:
            ws.random_()              # eager work that leaves other contents
        torch.cuda.synchronize()
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])


def step_buffers(n, heads, group, dim, bs, n_blocks, width, budget, dtype):
    F, hq = heads * dim, heads * group
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device=DEV)  # noqa: E731
    b = dict(k=z(n_blocks, bs, F, t=TORCH[dtype]), v=z(n_blocks, bs, F, t=TORCH[dtype]), bounds=z(n_blocks, 2, F, t=TORCH[dtype]),
             table=z(n, width), old=z(n), new=z(n), free=z(n_blocks), ff=z(1), taken=z(1), starts=z(n + 1), slots=z(n + 2),
             status=z(n), word=z(1), rows=z(n + 2, (group + 2) * F, t=TORCH[dtype]), blocks=z(n, heads, budget),
             out=z(n, hq * dim, t=TORCH[dtype]), dense=z(n, hq * dim, t=TORCH[dtype]), lse=z(n, hq, t=torch.float32))
    b["pages"] = K.make_pages(b["k"], b["v"], n_blocks, bs, heads, dim, dtype)
    b["req"] = K.make_requests(b["table"], width, b["new"], n, status=b["status"])
    b["plan"] = K.make_page_plan(b["old"], b["new"], n, bs, b["free"], n_blocks, n_blocks, b["table"], width, b["slots"], n + 2,
                                 free_from=b["ff"], starts=b["starts"], taken=b["taken"], status=b["status"])
    # a token's row: queries, key, value
    b["new_rows"] = K.make_page_rows(b["rows"][:, group * F:], b["rows"][:, (group + 1) * F:], n + 2, b["slots"], dtype,
                                     b["rows"].stride(0), b["rows"].stride(0), status=b["word"])
    scale = dim ** -0.5
    b["sparse"] = K.make_queries(b["rows"], b["out"], hq, scale, lse=b["lse"], q_stride=b["rows"].stride(0))
    b["full"] = K.make_queries(b["rows"], b["dense"], hq, scale, q_stride=b["rows"].stride(0))
    b["sel"] = K.make_selection(b["blocks"], budget, 1, 1)
    b["ws"] = torch.empty(K.kvtc_page_workspace_bytes(b["pages"], b["req"], b["sparse"], b["sel"]), dtype=torch.uint8, device=DEV)
    return b


def step(b, s):
    """One decoding step of a layer: every request's new token gets its place, its rows are written, the bounds of
    its page renewed, pages selected and attended to; attention over all of them beside it. The caller has set new."""
    K.kvtc_page_tables(b["plan"], s)
    K.kvtc_page_write(b["pages"], b["new_rows"], s)
    K.kvtc_page_bounds(b["pages"], b["req"], b["old"], b["bounds"], stream=s)
    K.kvtc_page_select(b["pages"], b["req"], b["sparse"], b["bounds"], b["sel"], b["ws"], stream=s)
    K.kvtc_page_attend(b["pages"], b["req"], b["sparse"], b["sel"], b["ws"], stream=s)
    K.kvtc_page_attend(b["pages"], b["req"], b["full"], None, b["ws"], stream=s)
    b["ff"].add_(b["taken"])
    b["old"].copy_(b["new"])


def check_step(b, n, heads, group, dim, bs, n_blocks, width, budget, dtype):
    shape = (n_blocks, bs, heads, dim)
    k, v = f64(b["k"]).reshape(shape), f64(b["v"]).reshape(shape)
    q = f64(b["rows"])[:n, :heads * group * dim].reshape(n, heads * group, dim)
    table, lens = b["table"].cpu().numpy(), b["new"].cpu().numpy()
    c = dict(q=torch.from_numpy(q), k=torch.from_numpy(k), v=torch.from_numpy(v), table=table, lens=lens, width=width, dim=dim, dtype=dtype)
    want, st = OP.select(q, f64(b["bounds"]).reshape(n_blocks, 2, heads, dim), table, lens, bs, n_blocks, width, heads, budget, 1, 1)
    assert np.array_equal(b["blocks"].cpu().numpy(), want)
    found, _ = OP.bounds(k, table, lens, width)
    for page, (lo, hi) in found.items():
        got = f64(b["bounds"])[page]
        assert np.array_equal(got[0], lo) and np.array_equal(got[1], hi)
    check_attend(c, dim ** -0.5, b["out"].cpu(), b["lse"].cpu(), blocks=want)
    _, lse, _, _ = OP.attend(q, k, v, table, lens, width, dim ** -0.5)
    check_attend(c, dim ** -0.5, b["dense"].cpu(), torch.from_numpy(lse))
    assert not b["status"].cpu().numpy().any() and int(b["word"]) == 0


@pytest.mark.parametrize("dtype,heads,group,dim,bs", [(BF16, 2, 4, 64, 4), (F32, 1, 2, 64, 16)])
def test_decoding_steps_eager_and_captured(dtype, heads, group, dim, bs):
    """The same steps eagerly and as replays of one graph, with eager work and synchronizations between the replays:
    equal bits after every step, checked against the oracle at some of them."""
    n, n_blocks, width, budget = 3, 64, 12, 5
    sizes = (n, heads, group, dim, bs, n_blocks, width, budget, dtype)
    eager, cap = step_buffers(*sizes), step_buffers(*sizes)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    order = torch.randperm(n_blocks, generator=g, device=DEV).to(torch.int32)
    for b in (eager, cap):
        b["free"].copy_(order)
        b["rows"].normal_()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):      # one step outside the graph first, undone by the reset below
        cap["new"].fill_(1)
        step(cap, side)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step(cap, side)
    for x in ("k", "v", "bounds", "table", "old", "new", "ff", "out", "dense", "lse"):
        cap[x].zero_()
    for t in range(14):
        rows = torch.randn(n + 2, (group + 2) * heads * dim, generator=g, device=DEV)
        grow = torch.tensor([1, 1 if t % 3 else 0, 1 if t > 4 else 0], dtype=torch.int32, device=DEV)
        for b in (eager, cap):
            b["rows"].copy_(rows)
            b["new"].add_(grow)
        step(eager, torch.cuda.current_stream())
        torch.cuda.synchronize()
        graph.replay()
        if t % 2:
            torch.cuda.synchronize()
        junk = torch.randn(1000, device=DEV).sum()
        torch.cuda.synchronize()
        assert float(junk) == float(junk)
        for x in ("k", "v", "bounds", "table", "slots", "starts", "taken", "ff", "blocks", "out", "dense", "lse"):
            assert torch.equal(eager[x], cap[x]), (t, x)
        if t in (0, 4, 13):
            check_step(cap, *sizes)


def test_restored_pages_then_decoding_steps():
    """Streams decoded by kvtc_decode into pages that kvtc_page_tables laid out, their bounds, then steps that append
    and attend: the two halves of a cache's life."""
    import oracle.kvtc_oracle as O
    w = synth.workload("odd3_bf16")
    art = oracle_artifact("odd3_bf16", [(0, 0), (0, 1)])
    dc = DevCodec(art.serialize())
    heads, group, dim, bs, lens = 3, 2, 64, 16, [500, 129]
    n, n_blocks, width, budget = 2, 48, 36, 6
    sizes = (n, heads, group, dim, bs, n_blocks, width, budget, BF16)
    b = step_buffers(*sizes)
    b["free"].copy_(torch.randperm(n_blocks, device=DEV).to(torch.int32))
    # the layout of the restored tokens: their slots are not needed, kvtc_decode takes the tables
    b["new"].copy_(dev(lens))
    slots = torch.empty(sum(lens), dtype=torch.int32, device=DEV)
    K.kvtc_page_tables(K.make_page_plan(None, b["new"], n, bs, b["free"], n_blocks, n_blocks, b["table"], width, slots, sum(lens),
                                        taken=b["taken"], status=b["status"]), torch.cuda.current_stream())
    b["ff"].copy_(b["taken"])
    jobs, keep = [], []
    for i, T in enumerate(lens):
        for kind, pages in ((0, b["k"]), (1, b["v"])):
            store = synth.storage(w, synth.gen_kv(w, 0, kind, synth.ROLE_EVAL, T, i))
            src = to_dev_bytes(O.encode(store, art.params, art.slots[(0, kind)], 0, kind).stream, 16)
            keep.append(src)
            jobs.append(K.make_job(0, kind, T, src, pages, pages.numel() * 2, b["table"][i], bs, n_blocks))
    st = dc.decode_jobs(jobs, BF16)
    assert not st.any()
    K.kvtc_page_bounds(b["pages"], b["req"], None, b["bounds"], stream=torch.cuda.current_stream())
    b["old"].copy_(b["new"])
    for t in range(20):
        b["rows"].normal_()
        b["new"].add_(1)
        step(b, torch.cuda.current_stream())
        torch.cuda.synchronize()
        if t in (0, 19):
            check_step(b, *sizes)
    # the decoded rows are where the slot map says
    flat = f64(b["k"]).reshape(-1, heads * dim)
    first = f64(b["k"]).reshape(n_blocks, bs, -1)[b["table"].cpu().numpy()[0, 0]]
    assert np.array_equal(flat[slots.cpu().numpy()[:bs]], first)
