"""GPU parity of packed-prompt attention (pkv_prompt_attention) against the
float64 oracle, within the bounds of attention_bounds; what a row may not
depend on; refusals."""

import numpy as np
import pytest
import torch

import attention_bounds as ab
from oracle import attention

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def inputs(lens, kv, hq, hkv, d, dtype, seed, device, fused=False, lead=0, tail=0):
    """Packed inputs with `lead` / `tail` rows of no sequence around them."""
    g = torch.Generator().manual_seed(seed)
    T, S = lead + sum(lens) + tail, lead + sum(kv) + tail
    t = TYPES[dtype]
    if fused:
        assert lens == kv
        x = torch.randn((T, (hq + 2 * hkv) * d), generator=g).to(t).to(device)
        q = x[:, :hq * d].unflatten(1, (hq, d))
        k = x[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        v = x[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    else:
        q, k, v = (torch.randn((n, h, d), generator=g).to(t).to(device) for n, h in ((T, hq), (S, hkv), (S, hkv)))
    qs = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32) + lead
    ks = np.concatenate([[0], np.cumsum(kv)]).astype(np.int32) + lead
    return q, k, v, qs, ks


def run(pkv, q, k, v, qs, ks, scale, workspace=True, fill=7.0):
    dev = q.device
    out = torch.full(q.shape, fill, dtype=q.dtype, device=dev)
    ws = None
    if workspace:
        n = pkv.pkv_prompt_attention_workspace_bytes(len(qs) - 1, q.shape[0], k.shape[0], q.shape[1], k.shape[1],
                                                     q.shape[2])
        ws = torch.full((n,), 255, dtype=torch.uint8, device=dev) if n else None  # NaN bits
    pkv.pkv_prompt_attention(q, k, v, torch.from_numpy(qs).to(dev), scale, out,
                             kv_start=None if ks is None else torch.from_numpy(ks).to(dev), workspace=ws)
    torch.cuda.synchronize()
    return out


def check(q, k, v, qs, ks, scale, got, fill=7.0, what=""):
    dtype, d = q.dtype, q.shape[2]
    qn, kn, vn = (x.float().cpu().numpy().astype(np.float64) for x in (q, k, v))
    want, want_abs = attention.prompt_attention(qn, kn, vn, qs, scale, ks)
    X = ab.score_bound(qn, kn, scale, qs, ks)
    v_sum = None
    if dtype == torch.float16:  # sum_t |v_t| over the sequence, per row and head
        G = qn.shape[1] // kn.shape[1]
        v_sum = np.zeros_like(qn)
        for b in range(len(qs) - 1):
            v_sum[qs[b]:qs[b + 1]] = np.repeat(np.abs(vn[ks[b]:ks[b + 1]]).sum(0), G, axis=0)[None]
    tol = ab.bound(want, want_abs, X, d, dtype, ab.half_step(dtype), v_sum)
    got = got.float().cpu().numpy()
    ab.assert_within(got[qs[0]:qs[-1]], want[qs[0]:qs[-1]], tol[qs[0]:qs[-1]], what)
    assert (got[:qs[0]] == fill).all() and (got[qs[-1]:] == fill).all(), "rows of no sequence were written"


@pytest.mark.gpu
@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 2), (6, 2), (8, 1)])
def test_ragged_lengths(pkv, cuda_dev, hq, hkv, d, dtype, workspace):
    lens = [1, 0, 2, 33, 127, 128, 129, 64, 300, 17]
    q, k, v, qs, ks = inputs(lens, lens, hq, hkv, d, dtype, hq + d, cuda_dev, lead=3, tail=5)
    out = run(pkv, q, k, v, qs, None, d ** -0.5, workspace)
    assert pkv.pkv_device_status() == 0
    check(q, k, v, qs, ks, d ** -0.5, out)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 15, 16, 31, 32, 33, 63, 64, 65, 255, 256, 257, 511, 513, 1025])
def test_single_prompts(pkv, cuda_dev, n):
    q, k, v, qs, ks = inputs([n], [n], 8, 2, 128, "bf16", n, cuda_dev)
    out = run(pkv, q, k, v, qs, None, 128 ** -0.5)
    assert pkv.pkv_device_status() == 0
    check(q, k, v, qs, ks, 128 ** -0.5, out, what="n %d" % n)


@pytest.mark.gpu
@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("lens,prefix", [([1], [0]), ([1], [5000]), ([7, 1, 60], [900, 128, 0]), ([40, 5], [4000, 3001]),
                                         ([130, 0, 20], [127, 300, 2500]), ([1] * 40, list(range(0, 4000, 100)))])
@pytest.mark.parametrize("hq,hkv,d,dtype", [(8, 2, 128, "bf16"), (8, 2, 64, "fp16"), (3, 1, 128, "fp16")])
def test_behind_a_prefix(pkv, cuda_dev, lens, prefix, hq, hkv, d, dtype, workspace):
    kv = [a + b for a, b in zip(lens, prefix)]
    q, k, v, qs, ks = inputs(lens, kv, hq, hkv, d, dtype, sum(kv), cuda_dev, tail=2)
    out = run(pkv, q, k, v, qs, ks, d ** -0.5, workspace)
    assert pkv.pkv_device_status() == 0
    check(q, k, v, qs, ks, d ** -0.5, out)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(5, 1), (7, 1), (12, 1), (48, 3), (128, 1), (100, 1), (10, 2)])
def test_group_sizes(pkv, cuda_dev, hq, hkv):
    lens = [40, 3, 201]
    q, k, v, qs, ks = inputs(lens, lens, hq, hkv, 64, "bf16", hq, cuda_dev)
    out = run(pkv, q, k, v, qs, None, 0.125)
    assert pkv.pkv_device_status() == 0
    check(q, k, v, qs, ks, 0.125, out, what="G %d" % (hq // hkv))


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.3, 0.0, -0.2, 1e-6])
def test_scales_of_any_sign(pkv, cuda_dev, scale):
    lens = [150, 20]
    q, k, v, qs, ks = inputs(lens, lens, 8, 2, 128, "bf16", 5, cuda_dev)
    out = run(pkv, q, k, v, qs, None, scale)
    check(q, k, v, qs, ks, scale, out, what="scale %g" % scale)


@pytest.mark.gpu
def test_strided_views_give_the_bits_of_dense_rows(pkv, cuda_dev):
    lens = [200, 33, 70]
    q, k, v, qs, ks = inputs(lens, lens, 8, 2, 128, "bf16", 9, cuda_dev, fused=True)
    a = run(pkv, q, k, v, qs, None, 0.09)
    b = run(pkv, q.contiguous(), k.contiguous(), v.contiguous(), qs, ks, 0.09)
    assert torch.equal(a, b)
    check(q, k, v, qs, ks, 0.09, a)


@pytest.mark.gpu
def test_growing_scores_raise_the_maximum(pkv, cuda_dev):
    """Keys whose scores grow along the prompt: every tile raises the running
    maximum by far more than its slack."""
    n = 700
    q, k, v, qs, ks = inputs([n], [n], 4, 1, 128, "bf16", 2, cuda_dev)
    q.fill_(0.5)
    k.copy_((torch.arange(n, device=cuda_dev) / 8.0)[:, None, None].expand(k.shape).to(k.dtype))
    out = run(pkv, q, k, v, qs, None, 0.25)
    check(q, k, v, qs, ks, 0.25, out)


@pytest.mark.gpu
@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (64, 4, 4)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_row_does_not_see_later_rows_or_other_sequences(pkv, cuda_dev, bad, d, hq, hkv):
    """Non-finite K and V at a position change the rows from it on, in its own
    sequence, and no other bit of the output."""
    lens = [100, 150, 90]
    q, k, v, qs, ks = inputs(lens, lens, hq, hkv, d, "fp16", 4, cuda_dev, lead=2, tail=3)
    base = run(pkv, q, k, v, qs, None, 0.1)
    check(q, k, v, qs, ks, 0.1, base)
    at = int(qs[1]) + 77
    k2, v2 = k.clone(), v.clone()
    v2[at, 0, 5] = bad
    v2[:2] = bad  # rows of no sequence
    k2[-3:] = bad
    v2[-3:] = bad
    got = run(pkv, q, k2, v2, qs, None, 0.1)
    hit = torch.zeros_like(base, dtype=torch.bool)
    hit[at:int(qs[2]), :hq // hkv, 5] = True
    assert torch.equal(got[~hit], base[~hit])
    x = got[hit]
    assert (torch.isnan(x) if bad != bad else (torch.isinf(x) & (x.sign() == (1 if bad > 0 else -1)))).all()
    k2 = k.clone()
    k2[at, 0, 5] = float("nan")
    got = run(pkv, q, k2, v, qs, None, 0.1)
    hit = torch.zeros_like(base, dtype=torch.bool)
    hit[at:int(qs[2]), :hq // hkv] = True
    assert torch.equal(got[~hit], base[~hit]) and torch.isnan(got[hit]).all()


@pytest.mark.gpu
def test_rows_without_keys_and_bad_ranges(pkv, cuda_dev):
    # more queries than K/V rows: zeros at negative positions, and a status bit
    q, k, v, qs, ks = inputs([50, 30], [20, 0], 8, 2, 64, "bf16", 6, cuda_dev)
    out = run(pkv, q, k, v, qs, ks, 0.125)
    assert pkv.pkv_device_status() == pkv.PKV_STATUS_BAD_CONTEXT
    check(q, k, v, qs, ks, 0.125, out)
    assert (out[:30] == 0).all() and (out[50:] == 0).all()
    # no K/V row at all
    out = run(pkv, q, k[:0], v[:0], qs, np.zeros(3, np.int32), 0.125)
    assert pkv.pkv_device_status() == pkv.PKV_STATUS_BAD_CONTEXT and (out == 0).all()
    # starts outside the rows or out of order: nothing outside is read or
    # written, and the call says so
    for bad_q, bad_k in (([0, 50, 1000], [0, 50, 80]), ([0, 50, 80], [0, 50, 1 << 30]), ([-7, 50, 80], [0, 50, 80]),
                         ([0, 60, 40], [0, 60, 80]), ([0, 50, 80], [40, 10, 80]), ([0, 50, 80], [-5, 50, 80])):
        q, k, v, _, _ = inputs([50, 30], [50, 30], 8, 2, 64, "bf16", 6, cuda_dev)
        run(pkv, q, k, v, np.array(bad_q, np.int32), np.array(bad_k, np.int32), 0.125)
        assert pkv.pkv_device_status() & pkv.PKV_STATUS_BAD_CONTEXT, (bad_q, bad_k)
    # all scores -inf: zeros
    q, k, v, qs, ks = inputs([8], [8], 1, 1, 64, "bf16", 6, cuda_dev)
    q.fill_(1.0)
    k.fill_(float("-inf"))
    out = run(pkv, q, k, v, qs, None, 1.0)
    assert (out == 0).all()


@pytest.mark.gpu
def test_nothing_to_do(pkv, cuda_dev):
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device=cuda_dev)
    out = torch.full_like(q, 3.0)
    one = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    pkv.pkv_prompt_attention(q, q, q, one, 1.0, out)  # batch 0
    pkv.pkv_prompt_attention(q[:0], q[:0], q[:0], torch.zeros(3, dtype=torch.int32, device=cuda_dev), 1.0, out[:0])
    pkv.pkv_prompt_attention(q, q, q, torch.tensor([2, 2, 2], dtype=torch.int32, device=cuda_dev), 1.0, out)
    torch.cuda.synchronize()
    assert (out == 3).all() and pkv.pkv_device_status() == 0


@pytest.mark.gpu
def test_repeats_streams_and_graph_replay_give_the_same_bits(pkv, cuda_dev):
    lens, prefix = [40, 300, 5], [900, 0, 2000]
    kv = [a + b for a, b in zip(lens, prefix)]
    q, k, v, qs, ks = inputs(lens, kv, 8, 2, 128, "bf16", 11, cuda_dev)
    first = run(pkv, q, k, v, qs, ks, 0.09)
    dq, dk = torch.from_numpy(qs).to(cuda_dev), torch.from_numpy(ks).to(cuda_dev)
    n = pkv.pkv_prompt_attention_workspace_bytes(3, q.shape[0], k.shape[0], 8, 2, 128)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device=cuda_dev)
    out = torch.zeros_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            pkv.pkv_prompt_attention(q, k, v, dq, 0.09, out, kv_start=dk, workspace=ws)
    s.synchronize()
    assert torch.equal(out, first)
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.pkv_prompt_attention(q, k, v, dq, 0.09, out, kv_start=dk, workspace=ws)
    q2 = torch.randn(q.shape, device=cuda_dev).to(q.dtype)
    want = run(pkv, q2, k, v, qs, ks, 0.09)
    keep = q.clone()
    for x, y in ((q2, want), (keep, first), (q2, want)):
        q.copy_(x)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)


@pytest.mark.gpu
@pytest.mark.parametrize("batch,top,hkv,d,dtype", [(40, 200, 8, 128, "bf16"), (31, 330, 8, 64, "fp16"), (70, 90, 4, 128, "fp16"),
                                                   (32, 130, 8, 64, "bf16")])
def test_more_rows_than_the_device_takes_at_once(pkv, cuda_dev, batch, top, hkv, d, dtype):
    # several (sequence, KV head) pairs of 256 rows for each SM, empty sequences
    # and prefixes among them
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, top, batch)
    lens[::7] = 0
    lens[1::7] = 1
    prefix = rng.integers(0, 150, batch) * (rng.random(batch) < 0.4)
    kv = (lens + prefix).tolist()
    lens = lens.tolist()
    q, k, v, qs, ks = inputs(lens, kv, 4 * hkv, hkv, d, dtype, batch, cuda_dev, lead=3, tail=130)
    out = run(pkv, q, k, v, qs, ks, 0.11)
    check(q, k, v, qs, ks, 0.11, out)
    assert torch.equal(out, run(pkv, q, k, v, qs, ks, 0.11))
    # a bad value in one sequence reaches its own later rows alone, not what the
    # same SM computes next
    b = int(np.argmax(lens))
    at = int(ks[b + 1]) - lens[b] // 2 - 1
    row = int(qs[b + 1]) - lens[b] // 2 - 1
    v2 = v.clone()
    v2[at, 1, 7] = float("nan")
    v2[int(ks[-1]):] = float("inf")  # rows of no sequence
    got = run(pkv, q, k, v2, qs, ks, 0.11)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[row:int(qs[b + 1]), 4:8, 7] = True
    assert torch.equal(got[~hit], out[~hit]) and torch.isnan(got[hit]).all()


@pytest.mark.gpu
def test_two_calls_at_once(pkv, cuda_dev):
    # both larger than the device: neither waits for the other's rows
    a = inputs([900] * 6, [900] * 6, 32, 8, 128, "bf16", 21, cuda_dev)
    b = inputs([70] * 50, [300] * 50, 32, 8, 64, "fp16", 22, cuda_dev)
    first = [run(pkv, *x, 0.1) for x in (a, b)]
    starts = [[torch.from_numpy(s).to(cuda_dev) for s in x[3:]] for x in (a, b)]
    outs = [torch.zeros_like(x[0]) for x in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for x, (qs, ks), out, s in zip((a, b), starts, outs, streams):
            with torch.cuda.stream(s):
                pkv.pkv_prompt_attention(*x[:3], qs, 0.1, out, kv_start=ks)
    torch.cuda.synchronize()
    assert pkv.pkv_device_status() == 0
    assert all(torch.equal(o, f) for o, f in zip(outs, first))


def test_refusals(pkv):
    L = pkv.lib
    ok = dict(q=16, k=16, v=16, qs=16, ks=None, batch=1, T=4, S=4, hq=8, hkv=2, d=128, sq=1024, sk=256, sv=256,
              scale=1.0, out=16, ws=None, wb=0, dtype=1)

    def call(**kw):
        a = dict(ok, **kw)
        return L.pkv_prompt_attention(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["batch"], a["T"], a["S"], a["hq"],
                                      a["hkv"], a["d"], a["sq"], a["sk"], a["sv"], a["scale"], a["out"], a["ws"],
                                      a["wb"], a["dtype"], None)

    for kw in (dict(hq=6, hkv=4), dict(batch=-1), dict(T=-1), dict(S=-1), dict(hkv=0), dict(dtype=5), dict(q=None),
               dict(k=None), dict(qs=None), dict(out=None), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(sq=1016), dict(sk=248), dict(sv=0)):
        assert call(**kw) == -1, kw
    for kw in (dict(d=96, sq=8192), dict(d=256, sq=8192, sk=8192, sv=8192), dict(hq=258, hkv=2, sq=1 << 20)):
        assert call(**kw) == -8, kw
    for kw in (dict(q=24), dict(k=20), dict(out=18), dict(sq=1028), dict(sk=260), dict(sv=257), dict(qs=18), dict(ks=18)):
        assert call(**kw) == -10, kw
    assert call(T=0, q=None, out=None) == 0 and call(batch=0) == 0
    with pytest.raises(pkv.PkvError):
        pkv.pkv_prompt_attention_workspace_bytes(1, 4, 4, 6, 4, 128)
    with pytest.raises(ValueError):
        x = torch.zeros((4, 64, 8), dtype=torch.bfloat16).transpose(1, 2)
        pkv.pkv_prompt_attention(x, x, x, torch.zeros(2, dtype=torch.int32), 1.0, torch.zeros((4, 8, 64)).bfloat16())
    with pytest.raises(TypeError):
        x = torch.zeros((4, 8, 64), dtype=torch.bfloat16)
        pkv.pkv_prompt_attention(x, x.half(), x, torch.zeros(2, dtype=torch.int32), 1.0, x.clone())
