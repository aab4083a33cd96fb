"""Compaction of sequences in the C++ block manager (through the C ABI, no
GPU) against the oracle's: tables, lengths, moves, reference counts and the
free stack; what may not happen to shared and cached blocks."""

import random

import numpy as np
import pytest

from oracle import allocator, kvcache


def _pair(pkv, nb, bs=16, seed=0):
    order = np.random.default_rng(seed).permutation(nb).astype(np.int32)
    return pkv.pkv_pool_create(nb, bs, order), allocator.KVCacheManager(nb, bs, order)


def _same(pkv, pool, ref):
    for s in ref.tables:
        assert list(pkv.pkv_seq_block_table(pool, s)) == ref.table(s)
        assert pkv.pkv_seq_len(pool, s) == ref.lens[s]
    assert pkv.pkv_pool_num_free(pool) == ref.pool.num_free()
    for b in range(ref.pool.num_blocks):
        assert pkv.pkv_block_refcount(pool, b) == ref.pool.ref[b]


def test_hand_worked_moves(pkv):
    # blocks of 4, handed out 0, 1, 2, ...: 10 tokens in blocks 0, 1, 2
    pool = pkv.pkv_pool_create(8, 4)
    s = pkv.pkv_seq_create(pool)
    pkv.pkv_seq_append(pool, s, 10)
    # rows 0..3 stay; position 4 is dropped, so 5..9 become 4..8 in blocks 3, 4
    src, dst = pkv.pkv_seq_compact(pool, s, [0, 1, 2, 3, 5, 6, 7, 8, 9])
    assert src.tolist() == [5, 6, 7, 8, 9] and dst.tolist() == [12, 13, 14, 15, 16]
    assert pkv.pkv_seq_block_table(pool, s).tolist() == [0, 3, 4]
    assert pkv.pkv_seq_len(pool, s) == 9 and pkv.pkv_pool_num_free(pool) == 5
    # blocks 1 and 2 were given back in that order: the next block is 2
    slots, pairs = pkv.pkv_seq_append(pool, s, 4)
    assert slots.tolist() == [17, 18, 19, 8] and pairs == []


def test_taking_back_the_last_tokens_moves_nothing(pkv):
    pool = pkv.pkv_pool_create(8, 4)
    s = pkv.pkv_seq_create(pool)
    pkv.pkv_seq_append(pool, s, 10)
    src, dst = pkv.pkv_seq_compact(pool, s, list(range(6)))  # two of block 1's rows stay
    assert len(src) == len(dst) == 0
    assert pkv.pkv_seq_block_table(pool, s).tolist() == [0, 1] and pkv.pkv_pool_num_free(pool) == 6
    slots, _ = pkv.pkv_seq_append(pool, s, 1)
    assert slots.tolist() == [6]
    # everything and nothing
    src, _ = pkv.pkv_seq_compact(pool, s, list(range(7)))
    assert len(src) == 0 and pkv.pkv_seq_len(pool, s) == 7
    src, _ = pkv.pkv_seq_compact(pool, s, [])
    assert len(src) == 0 and pkv.pkv_seq_len(pool, s) == 0 and pkv.pkv_pool_num_free(pool) == 8
    pkv.pkv_seq_append(pool, s, 5)  # an emptied sequence grows again


@pytest.mark.parametrize("seed", range(4))
def test_random_streams_match_the_oracle(pkv, seed):
    """Random create / append / fork / free / compact streams; the rows a
    model writes follow the moves, and every sequence still reads its own."""
    rng = random.Random(seed)
    bs = rng.choice([4, 8, 16])
    pool, ref = _pair(pkv, 60, bs, seed)
    rows = np.full((60, 1, bs, 1), -1.0)
    want = {}
    stamp = 0.0
    for _ in range(250):
        op = rng.choice(["create", "append", "append", "append", "fork", "compact", "compact", "free"])
        live = list(ref.tables)
        try:
            if op == "create" or not live:
                s = ref.create()
                assert pkv.pkv_seq_create(pool) == s
                want[s] = []
            elif op == "append":
                s, n = rng.choice(live), rng.randint(1, 3 * bs)
                slots, pairs = ref.append(s, n)
                got, gp = pkv.pkv_seq_append(pool, s, n)
                assert got.tolist() == slots and gp == pairs
                kvcache.copy_blocks([rows], pairs)
                for t in slots:
                    stamp += 1
                    rows[t // bs, 0, t % bs] = stamp
                    want[s].append(stamp)
            elif op == "fork":
                s = rng.choice(live)
                c = ref.fork(s)
                assert pkv.pkv_seq_fork(pool, s) == c
                want[c] = list(want[s])
            elif op == "free":
                s = rng.choice(live)
                ref.free(s)
                pkv.pkv_seq_free(pool, s)
                del want[s]
            else:
                ss = rng.sample(live, rng.randint(1, min(3, len(live))))
                keeps = [sorted(rng.sample(range(ref.lens[s]), rng.randint(0, ref.lens[s]))) for s in ss]
                if rng.random() < 0.3:
                    keeps[0] = list(range(len(keeps[0])))
                src, dst = ref.compact(ss, keeps)
                if len(ss) == 1 and rng.random() < 0.5:
                    gs, gd = pkv.pkv_seq_compact(pool, ss[0], keeps[0])
                else:
                    gs, gd = pkv.pkv_seq_compact_batch(pool, ss, keeps)
                assert gs.tolist() == src and gd.tolist() == dst
                # any order of the moves does: no destination block holds a source
                assert not {t // bs for t in dst} & {t // bs for t in src} and len(set(dst)) == len(dst)
                moves = list(zip(src, dst))
                rng.shuffle(moves)
                kvcache.move_rows([rows], [a for a, _ in moves], [b for _, b in moves], bs)
                for s, k in zip(ss, keeps):
                    want[s] = [want[s][t] for t in k]
        except allocator.OutOfBlocks:
            name = {"append": lambda: pkv.pkv_seq_append(pool, s, n),
                    "compact": lambda: pkv.pkv_seq_compact_batch(pool, ss, keeps)}[op]
            with pytest.raises(pkv.PkvError) as e:
                name()
            assert e.value.status == -2
        _same(pkv, pool, ref)
        for s, w in want.items():
            tab = ref.table(s)
            assert [rows[tab[i // bs], 0, i % bs, 0] for i in range(len(w))] == w
    pkv.pkv_pool_destroy(pool)


def test_cached_blocks_are_left_alone(pkv):
    pool = pkv.pkv_pool_create(16, 4)
    tokens = np.arange(12, dtype=np.int32)
    s = pkv.pkv_seq_create(pool)
    pkv.pkv_seq_append(pool, s, 12)
    assert pkv.pkv_prefix_register(pool, s, tokens) == 3
    cached = pkv.pkv_seq_block_table(pool, s).tolist()
    _, dst = pkv.pkv_seq_compact(pool, s, [1, 2, 3, 7, 11])
    assert not {int(t) // 4 for t in dst} & set(cached)
    t, n = pkv.pkv_prefix_match(pool, tokens)
    assert n == 12 and pkv.pkv_seq_block_table(pool, t).tolist() == cached


def test_refusals_change_nothing(pkv):
    pool, ref = _pair(pkv, 6, 4)
    s = ref.create()
    t = ref.create()
    assert pkv.pkv_seq_create(pool) == s and pkv.pkv_seq_create(pool) == t
    for x, n in ((s, 14), (t, 6)):
        ref.append(x, n)
        pkv.pkv_seq_append(pool, x, n)
    for keep in ([0, 0], [2, 1], [-1, 3], [0, 14], [14]):
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_seq_compact(pool, s, keep)
        assert e.value.status == -1
        _same(pkv, pool, ref)
    with pytest.raises(pkv.PkvError) as e:  # no free block for the one fresh block it takes
        pkv.pkv_seq_compact(pool, s, [1, 2])
    assert e.value.status == -2
    _same(pkv, pool, ref)
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_seq_compact_batch(pool, [s, s], [[0], [0]])
    assert e.value.status == -1
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_seq_compact(pool, 99, [0])
    assert e.value.status == -4
    _same(pkv, pool, ref)
    L = pkv.lib
    assert L.pkv_seq_compact(None, 0, None, 0, None, None, None) == -3
    assert L.pkv_seq_compact(pool, s, None, -1, None, None, None) == -1
    # a failing allocation (injected) leaves everything as it was
    pkv.pkv_seq_compact(pool, t, [0])
    ref.compact([t], [[0]])
    pkv.pkv_debug_fail_after(pool, 0)
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_seq_compact(pool, s, [1, 2])
    assert e.value.status == -2
    pkv.pkv_debug_fail_after(pool, -1)
    _same(pkv, pool, ref)


def test_move_rows_refusals(pkv):
    import ctypes
    L = pkv.lib
    ptr = (ctypes.c_void_p * 1)(16)
    odd = (ctypes.c_void_p * 1)(24)

    def call(pools=ptr, row=256, n_pools=1, src=16, dst=16, n=1, nb=4, h=2, bs=16):
        return L.pkv_move_rows(pools, (ctypes.c_int64 * 1)(row), n_pools, src, dst, n, nb, h, bs, None)

    assert call(n_pools=0) == -1 and call(n_pools=257) == -1 and call(row=0) == -1 and call(row=3) == -1
    assert call(n=-1) == -1 and call(nb=0) == -1 and call(h=0) == -1 and call(bs=0) == -1
    assert call(src=None) == -1 and call(pools=None) == -1
    assert call(row=1 << 17) == -8 and call(h=65536) == -8
    assert call(pools=odd) == -10 and call(src=20) == -10
    assert call(n=0, src=None, dst=None) == 0
