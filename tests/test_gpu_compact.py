"""GPU row moves (pkv_move_rows) against the oracle, bit for bit, and the
operators of a request run together: prompt attention, quantised append,
verify, rejected drafts taken back, eviction, decode."""

import numpy as np
import pytest
import torch

import attention_bounds as ab
from oracle import attention, kvcache

pytestmark = pytest.mark.gpu


def _pools(shapes, nb, hkv, bs, device, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(0, 256, (nb, hkv, bs, n), generator=g, dtype=torch.uint8).to(device) for n in shapes]


@pytest.mark.parametrize("rows", [[256, 256], [2, 64], [4, 128, 6, 10, 24], [2] * 9, [256] * 70, [2560, 40]])
@pytest.mark.parametrize("hkv,bs,n", [(1, 8, 1), (8, 16, 63), (3, 32, 64), (2, 16, 65), (5, 16, 300)])
def test_moves_match_the_oracle(pkv, cuda_dev, rows, hkv, bs, n):
    nb = 2 * (-(-n // bs)) + 4
    rng = np.random.default_rng(n)
    pools = _pools(rows, nb, hkv, bs, cuda_dev, n)
    half = nb // 2
    order = rng.permutation(nb)
    src = (order[:half][:, None] * bs + np.arange(bs)).reshape(-1)
    dst = (order[half:2 * half][:, None] * bs + np.arange(bs)).reshape(-1)
    src, dst = rng.permutation(src)[:n].astype(np.int64), rng.permutation(dst)[:n].astype(np.int64)
    if n > 10:
        src[3], dst[7] = -1, -5  # skipped
    want = [p.cpu().numpy().copy() for p in pools]
    kvcache.move_rows(want, src, dst, bs)
    ds, dd = torch.from_numpy(src).to(cuda_dev), torch.from_numpy(dst).to(cuda_dev)
    for _ in range(2):  # idempotent
        pkv.pkv_move_rows(pools, ds, dd)
    torch.cuda.synchronize()
    assert pkv.pkv_device_status() == 0
    for p, w in zip(pools, want):
        np.testing.assert_array_equal(p.cpu().numpy(), w)


def test_bad_slots_are_skipped_and_reported(pkv, cuda_dev):
    pools = _pools([128, 2], 8, 2, 16, cuda_dev, 1)
    want = [p.cpu().numpy().copy() for p in pools]
    src = np.array([0, 128, 5, 1 << 40, 6], np.int64)
    dst = np.array([64, 65, 128, 66, 67], np.int64)
    kvcache.move_rows(want, [0, 6], [64, 67])
    pkv.pkv_move_rows(pools, torch.from_numpy(src).to(cuda_dev), torch.from_numpy(dst).to(cuda_dev))
    torch.cuda.synchronize()
    assert pkv.pkv_device_status() == pkv.PKV_STATUS_BAD_SLOT
    for p, w in zip(pools, want):
        np.testing.assert_array_equal(p.cpu().numpy(), w)
    with pytest.raises(ValueError):
        pkv.pkv_move_rows([pools[0], pools[0][:, :1]], torch.zeros(1, dtype=torch.int64, device=cuda_dev),
                          torch.zeros(1, dtype=torch.int64, device=cuda_dev))


def test_row_offsets_past_32_bits(pkv, cuda_dev):
    """A pool of more than 2^32 bytes: the last blocks' rows."""
    nb, hkv, bs, row = 70000, 4, 16, 1024  # 4.6 GB
    pool = torch.zeros((nb, hkv, bs, row), dtype=torch.uint8, device=cuda_dev)
    last = torch.randint(0, 256, (1, hkv, bs, row), dtype=torch.uint8, device=cuda_dev)
    pool[nb - 1:] = last
    src = torch.arange(bs, dtype=torch.int64, device=cuda_dev) + (nb - 1) * bs
    pkv.pkv_move_rows([pool], src, src - bs)
    assert torch.equal(pool[nb - 2:nb - 1], last) and torch.equal(pool[nb - 1:], last)
    pkv.pkv_move_rows([pool], src, src - (nb - 1) * bs)
    assert torch.equal(pool[:1], last) and int(pool[1:nb - 2].max()) == 0


@pytest.mark.parametrize("mode", ["int4", "fp8"])
def test_a_request_from_prompt_to_eviction(pkv, cuda_dev, mode):
    """Two prompts are attended from their own rows and stored quantised; each
    sequence verifies 4 drafts, takes 2 back, evicts part of its middle, and
    decodes on: every step against 64 bits over the rows it should see."""
    dev, hq, hkv, d, t, ns = cuda_dev, 8, 2, 128, torch.bfloat16, 4
    scale = d ** -0.5
    g = torch.Generator().manual_seed(3)
    lens = [150, 77]
    NB = 80
    pool = pkv.pkv_pool_create(NB, 16, np.random.default_rng(2).permutation(NB).astype(np.int32))
    cb = d // 2 if mode == "int4" else d
    cache = {x + "_codes": torch.zeros((NB, hkv, 16, cb), dtype=torch.uint8, device=dev) for x in "kv"}
    names = ["scale", "zero"] if mode == "int4" else ["scale"]
    cache.update({x + "_" + n: torch.zeros((NB, hkv, 16, 1), dtype=torch.float16, device=dev) for x in "kv" for n in names})
    cache.update({"sink_" + x: torch.zeros((2, ns, hkv, d), dtype=t, device=dev) for x in "kv"})
    pools = [cache[x + "_" + n] for x in "kv" for n in ["codes"] + names]
    seqs = [pkv.pkv_seq_create(pool) for _ in lens]
    rows = [[np.zeros((0, hkv, d))] * 2 for _ in lens]

    def fresh(counts):
        q = torch.randn((sum(counts), hq, d), generator=g).to(t).to(dev)
        k, v = (torch.randn((sum(counts), hkv, d), generator=g).to(t).to(dev) for _ in range(2))
        return q, k, v

    def store(counts, k, v):
        at, slots, pos, idx = 0, [], [], []
        for b, n in enumerate(counts):
            s, pairs = pkv.pkv_seq_append(pool, seqs[b], n)
            assert not pairs
            slots.append(s)
            pos += range(len(rows[b][0]), len(rows[b][0]) + n)
            idx += [b] * n
            for i, x in enumerate((k, v)):
                rows[b][i] = np.concatenate([rows[b][i], x[at:at + n].float().cpu().numpy()])
            at += n
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        pkv.pkv_kv_append_quant(k, v, torch.from_numpy(np.concatenate(slots)).to(dev), i32(pos), i32(idx), cache, ns, mode, d)

    def inputs():
        mb = max(pkv.pkv_seq_num_blocks(pool, s) for s in seqs)
        tab, ctx = pkv.pkv_build_block_tables(pool, seqs, mb)
        assert ctx.tolist() == [len(r[0]) for r in rows]
        return torch.from_numpy(tab).to(dev), torch.from_numpy(ctx).to(dev)

    def check(got, q, counts, exact_rows, step, k_step, v_step):
        qn = q.float().cpu().numpy().astype(np.float64)
        at = 0
        for b, n in enumerate(counts):
            k, v = (x if exact_rows else kvcache.sequence_values(x.astype(np.float32), ns, mode, d) for x in rows[b])
            qb, st = qn[at:at + n], ([0, n], [0, len(k)])
            want, want_abs = attention.prompt_attention(qb, k, v, st[0], scale, st[1])
            tol = ab.bound(want, want_abs, ab.score_bound(qb, k, scale, *st), d, t, step,
                           np.abs(v).sum(0).repeat(hq // hkv, axis=0)[None], k_step, v_step)
            ab.assert_within(got[at:at + n].float().cpu().numpy(), want, tol, "sequence %d" % b)
            at += n

    # the prompts, from their own rows; then the quantised cache
    q, k, v = fresh(lens)
    qs = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device=dev)
    out = torch.empty_like(q)
    pkv.pkv_prompt_attention(q, k, v, qs, scale, out)
    store(lens, k, v)
    check(out, q, lens, True, 2.0 ** -8, 0.0, 0.0)
    u = 2.0 ** -11

    def verify(n):
        q, k, v = fresh([n, n])
        store([n, n], k, v)
        tab, ctx = inputs()
        out = torch.empty_like(q)
        qs = torch.tensor([0, n, 2 * n], dtype=torch.int32, device=dev)
        nb = pkv.pkv_multi_query_quant_workspace_bytes(2, hq, hkv, d, tab.shape[1], n)
        ws = torch.empty(max(nb, 16), dtype=torch.uint8, device=dev)
        pkv.pkv_paged_attention_multi_query_quant(q, qs, cache, ns, tab, ctx, scale, out, n, mode, workspace=ws)
        check(out, q, [n, n], False, u, 3 * u, 2 * u)

    verify(4)
    # two drafts rejected: nothing moves
    for b in range(2):
        n = len(rows[b][0]) - 2
        src, dst = pkv.pkv_seq_compact(pool, seqs[b], np.arange(n))
        assert len(src) == 0
        rows[b] = [x[:n] for x in rows[b]]
    verify(1)
    # the middle evicted: sinks and the last tokens stay
    keeps = [np.r_[0:20, 60:len(rows[0][0])], np.r_[0:ns, 10:len(rows[1][0]):3]]
    src, dst = pkv.pkv_seq_compact_batch(pool, seqs, keeps)
    pkv.pkv_move_rows(pools, torch.from_numpy(src).to(dev), torch.from_numpy(dst).to(dev))
    for b in range(2):
        rows[b] = [x[keeps[b]] for x in rows[b]]
    verify(3)
    verify(30)  # a slice
    assert pkv.pkv_device_status() == 0
    pkv.pkv_pool_destroy(pool)
