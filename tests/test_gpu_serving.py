"""The serving operators on the GPU against their definitions in 64 bits: the page plan, prompt
attention, shared-prefix decode, and a run of them together."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.serving_helpers import Pool, check_close, plan_reference  # noqa: E402

FMTS = ["q8_0", "q4_0", "lut4", "nvfp4"]


def dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=dtype)).cuda()


def tables(rng, num_pages, page_size, lens):
    """A page table of distinct random pages for sequences of the given lengths."""
    pages = [-(-int(n) // page_size) for n in lens]
    order = rng.permutation(num_pages)
    assert sum(pages) <= num_pages
    table = np.full((len(lens), max(1, max(pages))), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    return table, order[at:]


# ------------------------------------------------------------------ the plan

def run_plan(batch, ps, num_pages, max_pages, max_tokens, lens, new, free, count, table, planner=None, in_place=False):
    import quantized_kv_cache_split_b200 as K
    p = planner or K.PagePlanner(batch, ps, num_pages, max_pages, max_tokens)
    t = dev(table)
    f = dev(free)
    if in_place:
        p.seq_lens.copy_(dev(lens))
        p.free_count.fill_(count)
        p.step(dev(new), t, p.seq_lens, f, p.free_count)
    else:
        p.step(dev(new), t, dev(lens), f, dev([count]))
    torch.cuda.synchronize()
    return p, t.cpu().numpy(), f.cpu().numpy()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,ps,max_old,max_new,ended,max_tokens", [
    (1, 64, 0, 1, 0.0, 1), (1, 64, 64, 1, 0.0, 4), (3, 64, 200, 129, 0.0, 1000), (5, 192, 500, 0, 0.5, 3),
    (33, 128, 1000, 300, 0.3, 9901), (256, 64, 5000, 1, 0.0, 256), (1023, 64, 300, 40, 0.2, 40961),
    (1024, 64, 64, 65, 0.1, 70001), (61, 64, 3, 4000, 0.0, 244001)])
def test_plan_step(batch, ps, max_old, max_new, ended, max_tokens, in_place):
    rng = np.random.Generator(np.random.PCG64(batch + max_new))
    lens = rng.integers(0, max_old + 1, batch)
    new = rng.integers(0, max_new + 1, batch)
    new[rng.random(batch) < ended] = -1
    lens[0], new[0] = max_old, max_new  # the table's last column
    max_pages = -(-(max_old + max_new) // ps) or 1
    num_pages = batch * max_pages + 7
    table, rest = tables(rng, num_pages, ps, lens)
    wide = np.full((batch, max_pages), -1, dtype=np.int32)
    wide[:, :table.shape[1]] = table[:, :max_pages]
    free = np.full(num_pages, -5, dtype=np.int32)
    free[:len(rest)] = rest
    want = plan_reference(lens, new, free, len(rest), wide, ps, max_tokens)
    p, t, f = run_plan(batch, ps, num_pages, max_pages, max_tokens, lens, new, free, len(rest), wide, in_place=in_place)
    assert p.device_flags() == 0
    assert np.array_equal(t, want["table"])
    assert int(p.free_count) == len(want["stack"]) and np.array_equal(f[:len(want["stack"])], want["stack"])
    assert np.array_equal(p.seq_lens.cpu().numpy(), want["lens"])
    assert np.array_equal(p.token_offsets.cpu().numpy(), want["offsets"])
    assert np.array_equal(p.slots.cpu().numpy(), want["slots"])
    assert np.array_equal(p.positions.cpu().numpy(), want["positions"])


@pytest.mark.parametrize("max_tokens", [64, 20000])  # one CTA, and a cluster
@pytest.mark.parametrize("what,flag", [
    ("short", "KVQ_FLAG_NO_PAGES"), ("slots", "KVQ_FLAG_NO_SLOTS"), ("negative", "KVQ_FLAG_BAD_SEQLEN"),
    ("new", "KVQ_FLAG_BAD_SEQLEN"), ("long", "KVQ_FLAG_BAD_SEQLEN"), ("count", "KVQ_FLAG_BAD_PAGE"),
    ("free_id", "KVQ_FLAG_BAD_PAGE"), ("ended_id", "KVQ_FLAG_BAD_PAGE"), ("tail_id", "KVQ_FLAG_BAD_PAGE"),
    ("twice", "KVQ_FLAG_BAD_PAGE")])
def test_plan_step_refuses_and_changes_nothing(what, flag, max_tokens):
    import quantized_kv_cache_split_b200 as K
    lens, new = np.array([70, 10, 64, 0]), np.array([60, 1, 1, -1])
    table = np.array([[1, 2, -1], [3, -1, -1], [4, -1, -1], [-1, -1, -1]], dtype=np.int32)
    num_pages, free, count = 12, np.array([5, 6, 7, 8, 0, 0, 0, 0, 0, 0, 0, 0]), 4
    if what == "short":
        count = 1
    elif what == "slots":
        new[1] = 60
        max_tokens = 100
    elif what == "negative":
        lens[1] = -1
    elif what == "new":
        new[1] = -2
    elif what == "long":
        new[2] = 129
    elif what == "count":
        count = 13
    elif what == "free_id":
        free[3] = 12
    elif what == "ended_id":
        new[0], table[0, 1] = -1, -7
    elif what == "tail_id":
        table[1, 0] = 12
    elif what == "twice":
        new[0], num_pages = -1, 5   # more pages than the pool has
        free[:4] = [0, 1, 2, 3]
    p, t, f = run_plan(4, 64, num_pages, 3, max_tokens, lens, new, free, count, table)
    assert p.device_flags() == getattr(K, flag)
    assert np.array_equal(t, table)
    assert np.array_equal(f[:min(count, len(f))], free[:min(count, len(f))])
    assert int(p.free_count) == count and np.array_equal(p.seq_lens.cpu().numpy(), lens)
    assert not p.token_offsets.any() and bool((p.slots == -1).all()) and not p.positions.any()


# ------------------------------------------------------------------ prompt attention

def run_prompt(pool, G, old, new, *, causal=True, sm_scale=None, half=True, pad=0, max_extra=0, poison=True,
               with_table=True):
    """Every request's tokens against the definition; returns the relative error."""
    old, new = np.asarray(old), np.asarray(new)
    lens, hq = old + new, pool.hkv * G
    lens = np.maximum(lens, 0)
    if with_table:
        table, _ = tables(pool.rng, pool.num_pages, pool.ps, lens)
    else:
        width = pool.num_pages // len(lens)
        table = np.arange(len(lens) * width, dtype=np.int32).reshape(len(lens), width)
    total = int(new.sum())
    q = pool.queries(total + pad, hq)
    sm = 1.0 / math.sqrt(pool.D) if sm_scale is None else sm_scale
    offsets = np.concatenate(([0], np.cumsum(new)))
    owned = [pool.slots_of(table[b], lens[b]) for b in range(len(lens))]
    if poison:
        free = np.setdiff1d(np.arange(pool.num_pages * pool.ps), np.concatenate(owned))
        near = np.concatenate([pool.slots_of(table[b], min(-(-int(lens[b]) // pool.ps) * pool.ps, int(lens[b]) + 70))[lens[b]:]
                               for b in range(len(lens))]) if with_table else free[:0]
        pool.poison(np.concatenate((near, free[:50])).astype(np.int64))
    dtype = torch.float16 if half else torch.float32
    out = torch.full((total + pad, hq, pool.D), 7.0, dtype=dtype, device="cuda")
    got = pool.cache.prompt_attention(dev(q, np.float16), dev(offsets), dev(lens), int(lens.max()) + max_extra,
                                      dev(table) if with_table else None, table.shape[1], causal=causal,
                                      sm_scale=sm_scale, out=out).cpu().numpy()
    assert pool.cache.device_flags() == 0
    assert (got[total:] == 7.0).all()  # padding rows keep what the buffer held
    want, bound = np.zeros((total, hq, pool.D)), np.zeros((total, hq, pool.D))
    for b in range(len(lens)):
        for i in range(new[b]):
            seen = max(0, lens[b] - new[b] + i + 1) if causal else lens[b]
            want[offsets[b] + i], bound[offsets[b] + i] = pool.attend(q[offsets[b] + i], owned[b][:seen], sm)
    return check_close(got[:total], want, bound, half) if total else 0.0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_ragged(fmt, D):
    # lengths around the tile and page borders, requests without tokens, single tokens
    pool = Pool(fmt, D, 2, 64, 60, seed=1)
    err = run_prompt(pool, 4, [0, 63, 64, 0, 127, 128, 200, 5, 500], [1, 1, 64, 0, 2, 129, 57, 0, 33], pad=5)
    assert err < 2e-3


@pytest.mark.parametrize("G,hkv", [(1, 1), (3, 2), (5, 1), (7, 3), (8, 1)])
@pytest.mark.parametrize("page_size", [64, 192])
def test_prompt_heads_and_pages(G, hkv, page_size):
    # row tiles that end inside a token's heads; more than one row tile per request
    pool = Pool("q4_0", 128, hkv, page_size, 16, seed=2)
    run_prompt(pool, G, [0, 300], [131, 70])


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("fmt", ["q8_0", "lut4"])
def test_prompt_long_context_splits(fmt, half):
    # few rows over many positions: the positions are split and merged
    pool = Pool(fmt, 64, 1, 64, 110, seed=3)
    run_prompt(pool, 8, [5000, 1500], [3, 9], half=half, max_extra=1000)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_few_rows(fmt, D):
    # requests of a token or a few (at most 16 rows), beside one with more and one without any
    pool = Pool(fmt, D, 2, 64, 60, seed=20)
    run_prompt(pool, 4, [0, 63, 700, 64, 500, 10, 1, 127, 0, 300], [1, 4, 2, 0, 4, 9, 3, 1, 2, 4], pad=3)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("G,new", [(8, [1, 1, 1, 1]), (1, [8, 1, 5, 0]), (5, [3, 3, 3, 1]), (7, [1, 1, 1, 1])])
def test_prompt_few_rows_heads(G, new, causal):
    # single-token decode through prompt attention; tokens whose heads straddle 8-row tiles
    pool = Pool("q8_0", 128, 1, 64, 60, seed=21)
    run_prompt(pool, G, [1500, 0, 333, 1000], new, causal=causal)


def test_prompt_few_rows_without_positions():
    pool = Pool("q4_0", 64, 2, 64, 10, seed=22)
    run_prompt(pool, 4, [-2, -1, 20], [3, 1, 2])


def test_prompt_one_request_many_tokens():
    pool = Pool("q8_0", 128, 1, 64, 12, seed=4)
    run_prompt(pool, 2, [0], [700])


def test_prompt_not_causal():
    pool = Pool("nvfp4", 128, 2, 64, 30, seed=5)
    run_prompt(pool, 3, [0, 400, 10], [150, 20, 1], causal=False)


def test_prompt_rows_without_positions_are_zero():
    # more tokens than positions: the first ones see nothing; a sequence without any position
    pool = Pool("q4_0", 64, 2, 64, 10, seed=6)
    run_prompt(pool, 4, [-40, -3, 20], [100, 3, 2])
    run_prompt(pool, 4, [-40, -30], [40, 30])


@pytest.mark.parametrize("sm_scale", [-0.05, 0.0, 0.4])
@pytest.mark.parametrize("fmt", ["q4_0", "lut4"])
def test_prompt_scale_of_any_sign(fmt, sm_scale):
    pool = Pool(fmt, 64, 1, 64, 10, seed=7)
    run_prompt(pool, 4, [100, 0], [40, 20], sm_scale=sm_scale)


def test_prompt_without_page_table():
    pool = Pool("q8_0", 64, 2, 128, 8, seed=8)
    run_prompt(pool, 2, [100, 300], [30, 5], with_table=False, poison=False)


@pytest.mark.parametrize("fmt", FMTS)
def test_prompt_largest_values(fmt):
    # values at the edge of fp16: no code * scale may overflow, and equal keys give the mean
    import quantized_kv_cache_split_b200 as K
    pool = Pool(fmt, 128, 1, 64, 4, seed=9)
    big = 65504.0 if fmt != "lut4" else 5700.0   # lut4: the norm of the vector is fp16
    v = np.full((200, 1, 128), big, dtype=np.float16)
    v[::2] = -v[::2]
    k = np.zeros((200, 1, 128), dtype=np.float16)
    slots = dev(np.arange(200))
    pool.cache.write(dev(k, np.float16), dev(v, np.float16), slots)
    pool.k, pool.v = pool.values("k"), pool.values("v")
    out = pool.cache.prompt_attention(dev(pool.queries(1, 2), np.float16), dev([0, 1]), dev([200]), 256, dev([[0, 1, 2, 3]]),
                                      4).cpu().numpy()
    want, bound = pool.attend(pool.queries(1, 2)[0], np.arange(200), 1 / math.sqrt(128))
    check_close(out[0], want, bound, False)
    assert K is not None


def test_prompt_bad_pages_and_lengths_set_flags():
    import quantized_kv_cache_split_b200 as K
    pool = Pool("q8_0", 128, 1, 64, 8, seed=10)
    q = dev(pool.queries(4, 2), np.float16)
    ok = [[0, 1, 2]]
    for table, lens, offsets, flag in (
            ([[0, 8, 1]], [150], [0, 4], K.KVQ_FLAG_BAD_PAGE), ([[0, -1, 1]], [150], [0, 4], K.KVQ_FLAG_BAD_PAGE),
            (ok, [-1], [0, 4], K.KVQ_FLAG_BAD_SEQLEN), (ok, [193], [0, 4], K.KVQ_FLAG_BAD_SEQLEN),
            (ok, [150], [0, 5], K.KVQ_FLAG_BAD_SEQLEN), (ok, [150], [-1, 3], K.KVQ_FLAG_BAD_SEQLEN),
            (ok, [150], [3, 1], K.KVQ_FLAG_BAD_SEQLEN)):
        cache = K.QuantizedKVCache("q8_0", 128, 1, 64, 8)
        cache.prompt_attention(q, dev(offsets), dev(lens), 192, dev(table), 3)
        assert cache.device_flags() == flag, (table, lens, offsets)


# ------------------------------------------------------------------ shared prefixes

def run_prefix(pool, G, prefix, groups, own, *, half=True, sm_scale=None, extra=(0, 0), offsets=True, poison=True):
    """groups: requests per group, with leading requests outside every group as groups[0] < 0."""
    lead = -groups[0] if groups[0] < 0 else 0
    sizes = groups[1:] if lead else groups
    off = lead + np.concatenate(([0], np.cumsum(sizes)))
    B, hq = len(own), pool.hkv * G
    table, _ = tables(pool.rng, pool.num_pages, pool.ps, list(own) + list(prefix))
    own_slots = [pool.slots_of(table[b], own[b]) for b in range(B)]
    pre_slots = [pool.slots_of(table[B + g], prefix[g]) for g in range(len(prefix))]
    if poison:
        used = np.concatenate(own_slots + pre_slots)
        whole = np.concatenate([pool.slots_of(table[i], -(-int(n) // pool.ps) * pool.ps)
                                for i, n in enumerate(list(own) + list(prefix))])
        pool.poison(np.setdiff1d(whole, used)[:300])
    q = pool.queries(B, hq)
    sm = 1.0 / math.sqrt(pool.D) if sm_scale is None else sm_scale
    got = pool.cache.prefix_attention(
        dev(q, np.float16), dev(table[B:]), dev(prefix), max(prefix) + extra[0], dev(own), max(own) + extra[1],
        dev(table[:B]), table.shape[1], group_offsets=dev(off) if offsets else None, sm_scale=sm_scale,
        out_dtype=torch.float16 if half else torch.float32).cpu().numpy()
    assert pool.cache.device_flags() == 0
    want, bound = np.zeros((B, hq, pool.D)), np.zeros((B, hq, pool.D))
    for b in range(B):
        g = [i for i in range(len(sizes)) if off[i] <= b < off[i + 1]]
        slots = np.concatenate(([pre_slots[g[0]]] if g else []) + [own_slots[b]]).astype(np.int64)
        want[b], bound[b] = pool.attend(q[b], slots, sm)
    return check_close(got, want, bound, half)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
def test_prefix_one_group(fmt, D):
    pool = Pool(fmt, D, 2, 64, 60, seed=11)
    err = run_prefix(pool, 4, [1500], [9], [1, 64, 65, 130, 7, 300, 63, 2, 129], offsets=False)
    assert err < 2e-3


@pytest.mark.parametrize("G,hkv,B", [(1, 1, 1), (8, 1, 40), (5, 2, 60), (8, 3, 33), (3, 1, 86)])
def test_prefix_rows(G, hkv, B):
    # one row, one row tile, both row tiles, several units with a ragged end
    pool = Pool("q8_0", 64, hkv, 64, 16 + 2 * B, seed=12)
    run_prefix(pool, G, [777], [B], list(pool.rng.integers(0, 100, B)))


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("fmt", ["q4_0", "lut4"])
def test_prefix_groups(fmt, half):
    # ragged groups, one of them empty, one without a prefix, requests outside every group,
    # requests without own positions, one without any position at all
    pool = Pool(fmt, 128, 2, 64, 80, seed=13)
    run_prefix(pool, 3, [640, 100, 0, 65, 1999], [-2, 3, 0, 2, 1, 6], [5, 0, 40, 0, 129, 0, 3, 1, 1, 64, 0, 200, 10, 11, 0],
               half=half, extra=(100, 50))


def test_prefix_long():
    pool = Pool("nvfp4", 128, 1, 128, 100, seed=14)
    run_prefix(pool, 8, [9999], [20], [10] * 20)


def test_prefix_without_own_positions():
    pool = Pool("q4_0", 64, 2, 64, 20, seed=15)
    run_prefix(pool, 2, [800], [5], [0] * 5)


def test_prefix_no_own_positions_anywhere():
    # max_seq_len 0: requests outside every group have no position at all and get zeros
    pool = Pool("lut4", 64, 1, 64, 12, seed=23)
    q = dev(pool.queries(4, 2), np.float16)
    out = torch.full((4, 2, 64), 3.0, device="cuda")
    pool.cache.prefix_attention(q, dev([[5, 6, 7]]), dev([150]), 192, dev([0, 0, 0, 0]), 0, None, 1,
                                group_offsets=dev([1, 3]), out=out)
    got = out.cpu().numpy()
    assert not got[0].any() and not got[3].any()
    for b in (1, 2):
        want, bound = pool.attend(q.cpu().numpy()[b], pool.slots_of([5, 6, 7], 150), 1 / 8)
        check_close(got[b], want, bound, False)
    # and no prefix either
    pool.cache.prefix_attention(q, dev([[5, 6, 7]]), dev([0]), 0, dev([0, 0, 0, 0]), 0, None, 1, out=out)
    assert not out.any()


def test_prefix_40_groups():
    # more groups than lanes of a warp
    pool = Pool("q4_0", 64, 1, 64, 150, seed=24)
    prefix = list(pool.rng.integers(0, 130, 40))
    run_prefix(pool, 2, prefix, [1, 2] * 20, list(pool.rng.integers(0, 60, 60)))


def test_prompt_many_requests():
    pool = Pool("q8_0", 64, 1, 64, 200, seed=25)
    old, new = pool.rng.integers(0, 100, 70), pool.rng.integers(0, 40, 70)
    run_prompt(pool, 4, old, new)


@pytest.mark.parametrize("batch", [33, 300, 1024])
def test_prompt_batches_of_many_groups(batch):
    # the search for a block's group: many requests, some without tokens, some of several row tiles
    pool = Pool("q4_0", 64, 1, 64, 1100, seed=30)
    new = pool.rng.integers(0, 2, batch)
    new[batch // 2], new[batch // 3], new[-1] = 150, 65, 70
    old = np.where(pool.rng.random(batch) < 0.1, 40, 0)
    run_prompt(pool, 4, old, new, pad=2)


def test_prompt_many_groups_flag_bad_ones():
    import quantized_kv_cache_split_b200 as K
    pool = Pool("q8_0", 64, 1, 64, 8, seed=31)
    q = dev(pool.queries(40, 2), np.float16)
    off, lens = np.arange(41), np.full(40, 5)
    for what in ("len", "offset"):
        o, n = off.copy(), lens.copy()
        if what == "len":
            n[37] = 200
        else:
            o[21] = 0
        cache = K.QuantizedKVCache("q8_0", 64, 1, 64, 8)
        cache.prompt_attention(q, dev(o), dev(n), 128, dev(np.zeros((40, 2))), 2)
        assert cache.device_flags() == K.KVQ_FLAG_BAD_SEQLEN, what


def test_prompt_padding_before_the_first_request():
    pool = Pool("q8_0", 64, 1, 64, 8, seed=32)
    q = pool.queries(9, 2)
    out = torch.full((9, 2, 64), 5.0, device="cuda")
    pool.cache.prompt_attention(dev(q, np.float16), dev([3, 7]), dev([100]), 128, dev([[4, 2]]), 2, out=out)
    got = out.cpu().numpy()
    assert (got[:3] == 5.0).all() and (got[7:] == 5.0).all()
    for i in range(4):
        want, bound = pool.attend(q[3 + i], pool.slots_of([4, 2], 100)[:97 + i], 1 / 8)
        check_close(got[3 + i], want, bound, False)


@pytest.mark.parametrize("fmt", FMTS)
def test_prompt_growing_scores(fmt):
    # keys whose scores grow by far more than fp16's range from block to block, and fall again:
    # the maximum is raised many times
    pool = Pool(fmt, 128, 1, 64, 16, seed=26)
    n = 900
    grow = np.concatenate((np.linspace(0, 60, n // 2), np.linspace(60, -60, n - n // 2)))[:, None, None]
    k = (grow * pool.u / math.sqrt(128) + 0.1 * pool.rng.standard_normal((n, 1, 128))).astype(np.float16)
    v = pool.rng.standard_normal((n, 1, 128)).astype(np.float16)
    pool.cache.write(dev(k, np.float16), dev(v, np.float16), dev(np.arange(n)))
    pool.k, pool.v = pool.values("k"), pool.values("v")
    q = (pool.u + 0.1 * pool.rng.standard_normal((200, 2, 128))).astype(np.float16)
    out = pool.cache.prompt_attention(dev(q, np.float16), dev([0, 200]), dev([n]), n, dev([np.arange(16)]), 16).cpu().numpy()
    for i in (0, 1, 77, 199):
        want, bound = pool.attend(q[i], np.arange(n - 200 + i + 1), 1 / math.sqrt(128))
        check_close(out[i], want, bound, False)


def test_two_streams_at_once():
    # calls on two streams that overlap: a workspace each
    pool = Pool("q4_0", 128, 2, 64, 60, seed=27)
    qs = [dev(pool.queries(40, 8), np.float16) for _ in range(2)]
    tab = [dev([np.arange(30)]), dev([np.arange(30, 60)])]
    alone = [pool.cache.prefix_attention(qs[i], tab[i], dev([1900]), 1920, dev([0] * 40), 0).clone() for i in range(2)]
    own = dev([0] * 40)
    lens = dev([1900])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(pool.cache.prefix_attention(qs[i], tab[i], lens, 1920, own, 0))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, alone[i]) for o in outs[i])


def test_results_repeat_bit_for_bit():
    pool = Pool("q8_0", 128, 2, 64, 60, seed=28)
    q = dev(pool.queries(50, 8), np.float16)
    args = (q, dev([np.arange(40)]), dev([2500]), 2560, dev(pool.rng.integers(0, 20, 50)), 64,
            dev(np.tile(np.arange(40, 60), 3)[:50].reshape(50, 1)), 1)
    first = pool.cache.prefix_attention(*args)
    assert all(torch.equal(first, pool.cache.prefix_attention(*args)) for _ in range(5))


def test_methods_refuse_what_the_kernels_cannot_read():
    pool = Pool("q4_0", 128, 2, 64, 8, seed=29)
    c = pool.cache
    q = dev(pool.queries(4, 8), np.float16)
    off, lens, tab = dev([0, 4]), dev([100]), dev([[0, 1]])
    ok = lambda **kw: c.prompt_attention(**{**dict(q=q, token_offsets=off, seq_lens=lens, max_seq_len=128,  # noqa: E731
                                                  page_table=tab, max_pages=2), **kw})
    ok()
    wide = torch.zeros(4, 16, 128, dtype=torch.float16, device="cuda")
    for bad in (dict(q=wide[:, ::2]), dict(q=q.float()), dict(q=q[..., :64].contiguous()), dict(q=q.cpu()),
                dict(token_offsets=off.long()), dict(token_offsets=dev([0])), dict(seq_lens=lens.cpu()),
                dict(page_table=dev([[0, 1, 2, 3]])[:, ::2]), dict(max_pages=3), dict(out=torch.empty_like(q[:2])),
                dict(out=q.bfloat16()), dict(out_dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            ok(**bad)
    with pytest.raises(ValueError):
        c.prefix_attention(q, None, lens, 128, dev([0] * 4), 0)
    with pytest.raises(ValueError):
        c.prefix_attention(q, tab, lens, 128, dev([0] * 3), 0)


def test_prefix_and_decode_agree():
    # a request whose whole sequence is its own, or half of it the prefix: kvq_decode_attn's answer
    pool = Pool("q8_0", 128, 2, 64, 20, seed=16)
    q = dev(pool.queries(1, 8), np.float16)
    pages = pool.rng.permutation(20)[:10].astype(np.int32)
    whole = pool.cache.attention(q, dev([600]), 640, dev([pages]), 10, tau=0.0)
    for cut in (0, 5):
        part = pool.cache.prefix_attention(q, dev([np.concatenate((pages[:cut], pages[:1]))]), dev([64 * cut]), 640,
                                           dev([600 - 64 * cut]), 640, dev([np.concatenate((pages[cut:], pages[:cut]))]), 10)
        want, bound = pool.attend(q.cpu().numpy()[0], pool.slots_of(pages, 600), 1 / math.sqrt(128))
        check_close(part.cpu().numpy()[0], want, bound, False)
    check_close(whole.cpu().numpy()[0], want, bound, False)


# ------------------------------------------------------------------ together

def test_serving_run():
    """Plan, append, prompt attention, then decode steps on a shared prefix, then a request ends
    and its pages serve a new one: every answer against the definition on the cache's bytes."""
    import quantized_kv_cache_split_b200 as K
    ps, G, num_pages, mp, cap = 64, 4, 40, 8, 512
    pool = Pool("q4_0", 128, 2, ps, num_pages, seed=17)
    rng, B = pool.rng, 4
    prefix = np.arange(3, dtype=np.int32)                      # pages 0..2 hold the shared prefix
    plan = K.PagePlanner(B, ps, num_pages, mp, cap)
    table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
    free = dev(np.concatenate((np.arange(3, num_pages), [0, 0, 0])))
    plan.free_count.fill_(num_pages - 3)
    expect = np.zeros(B, dtype=np.int64)
    for new in ([100, 1, 65, 64], [1, 1, 1, 1], [1, 1, 1, -1], [1, 200, 1, 90]):
        plan.step(dev(new), table, plan.seq_lens, free, plan.free_count)
        k, v = (dev(rng.standard_normal((cap, 2, 128)), np.float16) for _ in range(2))
        pool.cache.write(k, v, plan.slots)                     # the padding is skipped
        torch.cuda.synchronize()
        pool.k, pool.v = pool.values("k"), pool.values("v")
        new = np.array(new)
        expect = np.where(new < 0, 0, expect + new)
        lens, tab = plan.seq_lens.cpu().numpy(), table.cpu().numpy()
        assert np.array_equal(lens, expect)
        own = [pool.slots_of(np.maximum(tab[b], 0), lens[b]) for b in range(B)]
        q = pool.queries(cap, 8)
        out = torch.zeros(cap, 8, 128, dtype=torch.float16, device="cuda")
        pool.cache.prompt_attention(dev(q, np.float16), plan.token_offsets, plan.seq_lens, mp * ps, table, mp, out=out)
        off = plan.token_offsets.cpu().numpy()
        for b in range(B):
            for i in range(off[b + 1] - off[b]):
                want, bound = pool.attend(q[off[b] + i], own[b][:lens[b] - (off[b + 1] - off[b]) + i + 1], 1 / math.sqrt(128))
                check_close(out[off[b] + i].cpu().numpy(), want, bound, True)
        assert not out[off[B]:].any()
        got = pool.cache.prefix_attention(dev(q[:B], np.float16), dev([prefix]), dev([150]), 192, plan.seq_lens, mp * ps,
                                          table, mp)
        for b in range(B):
            slots = np.concatenate((pool.slots_of(prefix, 150), own[b]))
            want, bound = pool.attend(q[b], slots, 1 / math.sqrt(128))
            check_close(got[b].cpu().numpy(), want, bound, False)
    assert plan.device_flags() == 0 and pool.cache.device_flags() == 0


def test_captured_step_replays_with_new_lengths():
    """One captured graph of plan, append, prompt and prefix attention on a side stream, replayed
    while the lengths on the GPU grow: the same answers as the calls made one by one."""
    import quantized_kv_cache_split_b200 as K
    ps, mp, cap, B = 64, 6, 40, 3
    pool = Pool("q8_0", 64, 1, ps, 24, seed=18)
    plan = K.PagePlanner(B, ps, 24, mp, cap)
    table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
    free = dev(np.arange(24))
    plan.free_count.fill_(20)                                  # pages 20..23: the prefix
    prefix, plens = dev([[20, 21, 22, 23]]), dev([250])
    new = dev([13, 1, 5])
    q = dev(pool.queries(cap, 2), np.float16)
    k, v = (dev(pool.rng.standard_normal((cap, 1, 64)), np.float16) for _ in range(2))
    out = torch.zeros(cap, 2, 64, dtype=torch.float16, device="cuda")
    dec = torch.zeros(B, 2, 64, dtype=torch.float16, device="cuda")

    def step():
        plan.step(new, table, plan.seq_lens, free, plan.free_count)
        pool.cache.write(k, v, plan.slots)
        pool.cache.prompt_attention(q, plan.token_offsets, plan.seq_lens, mp * ps, table, mp, out=out)
        pool.cache.prefix_attention(q[:B], prefix, plens, 256, plan.seq_lens, mp * ps, table, mp, out=dec)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    torch.cuda.synchronize()
    for turn in range(3):
        graph.replay()
        torch.cuda.synchronize()
        lens, tab, off = plan.seq_lens.cpu().numpy(), table.cpu().numpy(), plan.token_offsets.cpu().numpy()
        assert np.array_equal(lens, (turn + 2) * np.array([13, 1, 5]))
        pool.k, pool.v = pool.values("k"), pool.values("v")
        qn = q.cpu().numpy()
        for b in range(B):
            own = pool.slots_of(np.maximum(tab[b], 0), lens[b])
            for i in range(off[b + 1] - off[b]):
                want, bound = pool.attend(qn[off[b] + i], own[:lens[b] - (off[b + 1] - off[b]) + i + 1], 1 / 8)
                check_close(out[off[b] + i].cpu().numpy(), want, bound, True)
            want, bound = pool.attend(qn[b], np.concatenate((pool.slots_of([20, 21, 22, 23], 250), own)), 1 / 8)
            check_close(dec[b].cpu().numpy(), want, bound, True)
    assert plan.device_flags() == 0 and pool.cache.device_flags() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_write_skips_negative_slots(fmt):
    pool = Pool(fmt, 128, 2, 64, 3, seed=19)
    before = [getattr(pool.cache, p).clone() for p in ("k_codes", "k_scales", "v_codes", "v_scales")]
    x = dev(pool.rng.standard_normal((5, 2, 128)), np.float16)
    pool.cache.write(x, x, dev([-1, 70, -1, 3, -9]))
    torch.cuda.synchronize()
    for p, old in zip(("k_codes", "k_scales", "v_codes", "v_scales"), before):
        new = getattr(pool.cache, p).clone()
        assert not torch.equal(new.view(torch.uint8), old.view(torch.uint8))
        for s in (70, 3):
            new[s // 64, :, s % 64] = old[s // 64, :, s % 64]
        assert torch.equal(new.view(torch.uint8), old.view(torch.uint8))
