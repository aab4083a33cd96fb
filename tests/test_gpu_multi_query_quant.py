"""GPU parity of multi-query attention over the quantised cache
(pkv_paged_attention_multi_query_quant) against the float64 oracle over its own
dequantised values, within the bounds of attention_bounds; refusals."""

import numpy as np
import pytest
import torch

import attention_bounds as ab
from oracle import attention, kvcache

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


class Cache:
    pass


def build(pkv, lens, hq, hkv, d, dtype, mode, group, n_sink, window, seed, device, magnitude=1.0, rows_fn=None):
    """A shuffled quantised cache holding `lens` tokens per sequence, written
    by pkv_kv_append_quant; every slot never written holds NaN codes, scales
    and zero points."""
    c = Cache()
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // 16) for n in lens]
    NB = sum(need) + 5
    pool = pkv.pkv_pool_create(NB, 16, np.random.default_rng(seed).permutation(NB).astype(np.int32))
    cb, ng = (d // 2, d // group) if mode == "int4" else (d, 1)
    nan = float("nan")
    c.cache = {}
    for x in "kv":
        c.cache[x + "_codes"] = torch.full((NB, hkv, 16, cb), 0x7F, dtype=torch.uint8, device=device)
        c.cache[x + "_scale"] = torch.full((NB, hkv, 16, ng), nan, dtype=torch.float16, device=device)
        if mode == "int4":
            c.cache[x + "_zero"] = torch.full((NB, hkv, 16, ng), nan, dtype=torch.float16, device=device)
        if n_sink:
            c.cache["sink_" + x] = torch.full((len(lens), n_sink, hkv, d), nan, dtype=t, device=device)
        if window:
            c.cache["win_" + x] = torch.full((len(lens), window // 16 + 1, hkv, 16, d), nan, dtype=t, device=device)
    c.rows, seqs = [], []
    for b, n in enumerate(lens):
        seqs.append(pkv.pkv_seq_create(pool))
        k, v = (torch.randn((n, hkv, d), generator=g) * magnitude for _ in range(2))
        if rows_fn:
            rows_fn(b, k, v)
        k, v = k.to(t), v.to(t)
        c.rows.append((k.float().numpy(), v.float().numpy()))
        if n == 0:
            continue
        slots, _ = pkv.pkv_seq_append(pool, seqs[-1], n)
        pos = torch.arange(n, dtype=torch.int32, device=device)
        pkv.pkv_kv_append_quant(k.to(device), v.to(device), torch.from_numpy(slots).to(device), pos,
                                torch.full_like(pos, b), c.cache, n_sink, mode, group, window=window)
    c.max_blocks = max(max(need), 1)
    tables, ctx = pkv.pkv_build_block_tables(pool, seqs, c.max_blocks)
    c.tables, c.ctx = torch.from_numpy(tables).to(device), torch.from_numpy(ctx).to(device)
    c.lens, c.mode, c.group, c.n_sink, c.window = lens, mode, group, n_sink, window
    c.hq, c.hkv, c.d, c.t, c.device = hq, hkv, d, t, device
    pkv.pkv_pool_destroy(pool)
    torch.cuda.synchronize()
    return c


def queries(c, qlens, seed):
    q = torch.randn((sum(qlens), c.hq, c.d), generator=torch.Generator().manual_seed(seed + 100)).to(c.t)
    return q, np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)


def run(pkv, c, q, qs, scale, max_q=None, ctx=None, tables=None, tail=0, fill=7.0):
    dev = c.device
    max_q = max(1, int(np.diff(qs).max())) if max_q is None else max_q
    out = torch.full((q.shape[0] + tail,) + q.shape[1:], fill, dtype=q.dtype, device=dev)
    n = pkv.pkv_multi_query_quant_workspace_bytes(len(qs) - 1, c.hq, c.hkv, c.d, c.max_blocks, max_q)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=dev) if n else None  # NaN bits
    pkv.pkv_paged_attention_multi_query_quant(
        q.to(dev), torch.from_numpy(qs).to(dev), c.cache, c.n_sink, c.tables if tables is None else tables,
        c.ctx if ctx is None else ctx, scale, out, max_q, c.mode, group_size=c.group, workspace=ws, window=c.window)
    torch.cuda.synchronize()
    assert (out[q.shape[0]:] == fill).all()
    return out[:q.shape[0]]


def expected(c, q, qs, scale, seqs=None):
    """(want, bound) [T, Hq, D].  Against the dequantised values: the verify
    kernels multiply exact codes; their weights times the scale, and the
    queries, are rounded to fp16 (2^-11).  The slice kernel also rounds K and V
    values to fp16, in two steps (2 x 2^-11) of the value.  16-bit rows of a
    bf16 cache enter as bf16 weights (2^-8, twice for their residual: 2^-16)
    or as fp16."""
    qn = q.float().numpy().astype(np.float64)
    want, want_abs, X, v_sum = (np.zeros_like(qn) for _ in range(4))
    for b in range(len(qs) - 1) if seqs is None else seqs:
        k, v = (kvcache.sequence_values(x, c.n_sink, c.mode, c.group, c.window) for x in c.rows[b])
        r = slice(int(qs[b]), int(qs[b + 1]))
        if qs[b + 1] > qs[b]:
            want[r], want_abs[r] = attention.prompt_attention(qn[r], k, v, [0, qs[b + 1] - qs[b]], scale, [0, len(k)])
            X[r] = ab.score_bound(qn[r], k, scale, [0, qs[b + 1] - qs[b]], [0, len(k)])
            v_sum[r] = np.repeat(np.abs(v).sum(0), c.hq // c.hkv, axis=0)[None] if len(v) else 0
    step = 2.0 ** -11
    return want, ab.bound(want, want_abs, X, c.d, c.t, step, v_sum, k_step=3 * step, v_step=2 * step)


def check(c, q, qs, scale, got, what=""):
    want, tol = expected(c, q, qs, scale)
    ab.assert_within(got.float().cpu().numpy(), want, tol, what)


LAYOUTS = [("int4", 128, 128), ("int4", 64, 128), ("int4", 64, 64), ("fp8", 128, 128), ("fp8", 64, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("mode,group,d", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n_sink,window", [(0, 0), (4, 0), (8, 64), (16, 16)])
def test_layouts(pkv, cuda_dev, mode, group, d, dtype, n_sink, window):
    lens = [1, 16, 17, 33, 5, 300, 129, 64, 0, 80]
    qlens = [1, 3, 6, 6, 2, 6, 1, 4, 0, 5]
    c = build(pkv, lens, 8, 2, d, dtype, mode, group, n_sink, window, d + n_sink, cuda_dev)
    q, qs = queries(c, qlens, 1)
    got = run(pkv, c, q, qs, d ** -0.5, tail=3)
    assert pkv.pkv_device_status() == 0
    check(c, q, qs, d ** -0.5, got)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["int4", "fp8"])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (3, 1), (10, 2), (6, 1), (14, 2), (8, 1)])
@pytest.mark.parametrize("L", [1, 2, 3, 8])
def test_groups_and_query_counts(pkv, cuda_dev, mode, hq, hkv, L):
    lens = [L, 40, 500, 23]
    c = build(pkv, lens, hq, hkv, 128, "bf16", mode, 128, 4, 0, hq, cuda_dev)
    q, qs = queries(c, [L] * 4, L)
    got = run(pkv, c, q, qs, 0.09)
    assert pkv.pkv_device_status() == 0
    check(c, q, qs, 0.09, got)


@pytest.mark.gpu
@pytest.mark.parametrize("mode,group,d", LAYOUTS)
@pytest.mark.parametrize("n_sink,window,dtype", [(4, 0, "bf16"), (8, 128, "fp16"), (8, 32, "bf16"), (0, 0, "fp16")])
def test_slices(pkv, cuda_dev, mode, group, d, n_sink, window, dtype):
    lens = [300, 1000, 90, 128, 513]
    qlens = [130, 65, 90, 1, 257]
    c = build(pkv, lens, 8, 2, d, dtype, mode, group, n_sink, window, 3 + d, cuda_dev)
    q, qs = queries(c, qlens, 2)
    got = run(pkv, c, q, qs, d ** -0.5, tail=2)
    assert pkv.pkv_device_status() == 0
    check(c, q, qs, d ** -0.5, got)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (5, 1), (7, 1), (16, 2)])
@pytest.mark.parametrize("L", [25, 31, 32, 33, 128, 129])
def test_slice_groups(pkv, cuda_dev, hq, hkv, L):
    c = build(pkv, [L, 700, L + 13], hq, hkv, 128, "bf16", "int4", 128, 4, 0, L, cuda_dev)
    q, qs = queries(c, [L, min(L, 700), L], L)
    got = run(pkv, c, q, qs, 0.09)
    assert pkv.pkv_device_status() == 0
    check(c, q, qs, 0.09, got)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["int4", "fp8"])
@pytest.mark.parametrize("L", [5, 40])
@pytest.mark.parametrize("scale", [0.0, -0.1, 0.5])
def test_scales_of_any_sign(pkv, cuda_dev, mode, L, scale):
    c = build(pkv, [200, 60], 4, 1, 128, "bf16", mode, 128, 4, 32, 8, cuda_dev)
    q, qs = queries(c, [L, L], 3)
    got = run(pkv, c, q, qs, scale)
    check(c, q, qs, scale, got)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["int4", "fp8"])
@pytest.mark.parametrize("L", [4, 60])
def test_outliers_and_growing_scores(pkv, cuda_dev, mode, L):
    """Large V outliers (scales in the hundreds) and keys whose scores grow."""
    def rows(b, k, v):
        v[::7, 0, 3] = 4000.0
        v[5::11, 0, 70] = -4000.0
        k[:] = torch.linspace(0.0, 12.0, k.shape[0])[:, None, None]
        k[:, 0, 0] += 1.0

    c = build(pkv, [333, 150], 2, 1, 128, "fp16", mode, 128, 0, 0, 8, cuda_dev, rows_fn=rows)
    q, qs = queries(c, [L, L], 3)
    q.fill_(0.5)
    got = run(pkv, c, q, qs, 0.2)
    check(c, q, qs, 0.2, got)


@pytest.mark.gpu
@pytest.mark.parametrize("mode,group", [("int4", 64), ("fp8", 128)])
@pytest.mark.parametrize("window", [0, 64])
def test_one_query_equals_decode(pkv, cuda_dev, mode, group, window):
    """L = 1 is the quantised decode: the two kernels' outputs are within the
    same bound of the same values."""
    lens = [700, 33, 1, 250]
    c = build(pkv, lens, 8, 2, 128, "bf16", mode, group, 4, window, 21, cuda_dev)
    q, qs = queries(c, [1] * 4, 5)
    got = run(pkv, c, q, qs, 0.09)
    check(c, q, qs, 0.09, got)
    dec = torch.empty_like(got)
    n = pkv.pkv_decode_workspace_bytes(4, 8, 128, c.max_blocks)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device=cuda_dev)
    pkv.pkv_paged_attention_decode_quant(q.to(cuda_dev), c.cache, 4, c.tables, c.ctx, 0.09, dec, mode, group_size=group,
                                         workspace=ws, window=window)
    torch.cuda.synchronize()
    check(c, q, qs, 0.09, dec, "decode")


@pytest.mark.gpu
@pytest.mark.parametrize("L", [3, 30])
def test_a_row_does_not_see_later_rows(pkv, cuda_dev, L):
    """NaN in a later token's 16-bit and FP8 V row: rows before it keep their
    bits, rows from it on are NaN in that column."""
    n = 90
    for mode, window in (("fp8", 0), ("fp8", 32), ("int4", 32)):
        c0 = build(pkv, [n, 50], 4, 2, 128, "bf16", mode, 128, 4, window, 31, cuda_dev)
        q, qs = queries(c0, [L, L], 6)
        base = run(pkv, c0, q, qs, 0.09)
        check(c0, q, qs, 0.09, base)

        def rows(b, k, v):
            if b == 0:
                v[n - 2, 1, 9] = float("nan")

        c1 = build(pkv, [n, 50], 4, 2, 128, "bf16", mode, 128, 4, window, 31, cuda_dev, rows_fn=rows)
        got = run(pkv, c1, q, qs, 0.09)
        # the last two rows of sequence 0 see the token (KV head 1: query heads 2, 3)
        other = torch.ones_like(base, dtype=torch.bool)
        other[L - 2:L, 2:] = False
        assert torch.equal(got[other], base[other]), (mode, window)
        assert torch.isnan(got[L - 2:L, 2:, 9]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("L", [4, 50])
def test_bad_tables_and_contexts(pkv, cuda_dev, L):
    c = build(pkv, [200, 100, 60], 8, 2, 128, "bf16", "int4", 128, 4, 0, 41, cuda_dev)
    q, qs = queries(c, [L] * 3, 7)
    good = run(pkv, c, q, qs, 0.09)
    assert pkv.pkv_device_status() == 0
    for bad in (-1, 10 ** 6, 2 ** 31 - 1):
        t = c.tables.clone()
        t[1, 2] = bad
        got = run(pkv, c, q, qs, 0.09, tables=t)
        assert pkv.pkv_device_status() == pkv.PKV_STATUS_BAD_BLOCK
        assert torch.equal(got[:L], good[:L]) and torch.equal(got[2 * L:], good[2 * L:])
        assert torch.isfinite(got.float()).all()
    want, tol = expected(c, q, qs, 0.09)

    def others(got, rows):
        """The other sequences' rows: within the bound (another context moves
        the shares of the split, so not the same bits)."""
        ab.assert_within(got[rows].float().cpu().numpy(), want[rows], tol[rows])

    for bad in (-3, 2 ** 30, 16 * c.max_blocks + 1):
        ctx = c.ctx.clone()
        ctx[1] = bad
        got = run(pkv, c, q, qs, 0.09, ctx=ctx)
        assert pkv.pkv_device_status() & pkv.PKV_STATUS_BAD_CONTEXT
        others(got, slice(0, L))
        others(got, slice(2 * L, 3 * L))
        if bad < 0:
            assert (got[L:2 * L] == 0).all()
    # fewer tokens than queries: zeros at negative positions
    ctx = c.ctx.clone()
    ctx[2] = L - 2
    got = run(pkv, c, q, qs, 0.09, ctx=ctx)
    assert pkv.pkv_device_status() == pkv.PKV_STATUS_BAD_CONTEXT
    assert (got[2 * L:2 * L + 2] == 0).all()
    others(got, slice(0, 2 * L))
    # more queries than max_q_len: the first max_q_len rows only, the rest untouched
    got = run(pkv, c, q, qs, 0.09, max_q=L - 1)
    assert pkv.pkv_device_status() == pkv.PKV_STATUS_BAD_CONTEXT
    assert (got[L - 1] == 7).all() and (got[2 * L - 1] == 7).all()
    for b in range(3):
        others(got, slice(b * L, (b + 1) * L - 1))


@pytest.mark.gpu
@pytest.mark.parametrize("L", [6, 64])
def test_many_short_sequences(pkv, cuda_dev, L):
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(L, 200, size=120)]
    qlens = [int(x) for x in rng.integers(0, L + 1, size=120)]
    c = build(pkv, lens, 8, 2, 64, "bf16", "int4", 64, 4, 0, 51, cuda_dev)
    q, qs = queries(c, qlens, 8)
    got = run(pkv, c, q, qs, 0.125, max_q=L)
    assert pkv.pkv_device_status() == 0
    check(c, q, qs, 0.125, got)


@pytest.mark.gpu
@pytest.mark.parametrize("L", [6, 100])
def test_long_context_repeats_and_graph_replay(pkv, cuda_dev, L):
    c = build(pkv, [9000, 300], 8, 2, 128, "bf16", "int4", 64, 8, 128, 61, cuda_dev)
    q, qs = queries(c, [L, L], 9)
    first = run(pkv, c, q, qs, 0.09)
    check(c, q, qs, 0.09, first)
    n = pkv.pkv_multi_query_quant_workspace_bytes(2, 8, 2, 128, c.max_blocks, L)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device=cuda_dev)
    dq, dqs, out = q.to(cuda_dev), torch.from_numpy(qs).to(cuda_dev), torch.zeros_like(first)

    def call():
        pkv.pkv_paged_attention_multi_query_quant(dq, dqs, c.cache, 8, c.tables, c.ctx, 0.09, out, L, "int4",
                                                  group_size=64, workspace=ws, window=128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            call()
    s.synchronize()
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        out.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


def test_refusals(pkv):
    L = pkv.lib
    base = dict(q=16, qs=16, kc=16, ks=16, kz=16, vc=16, vs=16, vz=16, sk=16, sv=16, n_sink=4, wk=None, wv=None,
                window=0, tab=16, ctx=16, batch=2, hq=8, hkv=2, d=128, nb=10, bs=16, mb=4, mq=6, group=128, scale=1.0,
                out=16, ws=None, wb=0, qmode=1, dtype=1)

    def call(**kw):
        a = dict(base, **kw)
        return L.pkv_paged_attention_multi_query_quant(*[a[k] for k in base], None)

    for kw in (dict(batch=-1), dict(hq=6, hkv=4), dict(dtype=3), dict(qmode=0), dict(qmode=3), dict(q=None),
               dict(kz=None), dict(sk=None), dict(window=24), dict(window=32), dict(mq=-1), dict(nb=0), dict(mb=-1),
               dict(scale=float("nan")), dict(scale=float("-inf")), dict(n_sink=-1), dict(tab=None), dict(out=None)):
        assert call(**kw) == -1, kw
    for kw in (dict(d=96), dict(bs=8), dict(bs=32), dict(hq=18, hkv=2), dict(n_sink=17), dict(group=32),
               dict(batch=65536), dict(mb=1 << 27)):
        assert call(**kw) == -8, kw
    for kw in (dict(q=24), dict(kc=20), dict(vs=18), dict(sk=24), dict(out=8), dict(qs=18), dict(ctx=17)):
        assert call(**kw) == -10, kw
    assert call(batch=0, q=None) == 0 and call(mq=0, q=None) == 0
    with pytest.raises(pkv.PkvError):
        pkv.pkv_multi_query_quant_workspace_bytes(2, 8, 2, 128, 4, 6, block_size=8)
