"""Host-only checks of the serving calls: arguments are refused before anything is launched (the
pointers here are never dereferenced), workspace sizes, and the staging ring's barrier scheme."""
import random

import pytest

import quantized_kv_cache_split_b200 as K

FAKE = 1 << 20  # aligned dummy device pointer


def desc(fmt="q8_0", head_dim=128, num_kv_heads=4, page_size=64, num_pages=8, codebook=None, signs=None):
    return K.make_desc(fmt, head_dim, num_kv_heads, page_size, num_pages, codebook, signs)


# ------------------------------------------------------------------ the plan

def plan(**kw):
    a = dict(batch=4, page_size=64, num_pages=100, max_pages=10, max_tokens=64, seq_lens=FAKE, new_lens=FAKE,
             free_pages=FAKE, free_count=FAKE, page_table=FAKE, seq_lens_out=FAKE, free_count_out=FAKE,
             token_offsets=FAKE, slots=FAKE, positions=FAKE, workspace=FAKE, workspace_bytes=256)
    a.update(kw)
    return K.kvq_plan_step(*a.values(), stream=0, check=False)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), K.KVQ_ERR_INVALID_ARG), (dict(batch=1025), K.KVQ_ERR_UNSUPPORTED),
    (dict(page_size=63), K.KVQ_ERR_UNSUPPORTED), (dict(page_size=0), K.KVQ_ERR_UNSUPPORTED),
    (dict(num_pages=0), K.KVQ_ERR_INVALID_ARG), (dict(max_pages=0), K.KVQ_ERR_INVALID_ARG),
    (dict(max_tokens=-1), K.KVQ_ERR_INVALID_ARG), (dict(num_pages=1 << 26), K.KVQ_ERR_UNSUPPORTED),
    (dict(max_pages=1 << 26), K.KVQ_ERR_UNSUPPORTED), (dict(workspace_bytes=255), K.KVQ_ERR_WORKSPACE),
    (dict(slots=FAKE + 4), K.KVQ_ERR_INVALID_ARG), (dict(positions=FAKE + 8), K.KVQ_ERR_INVALID_ARG),
    (dict(workspace=FAKE + 4), K.KVQ_ERR_INVALID_ARG), (dict(batch=0), K.KVQ_OK)])
def test_plan_step_refusals(kw, code):
    assert plan(**kw) == code


@pytest.mark.parametrize("name", ["seq_lens", "new_lens", "free_pages", "free_count", "page_table", "seq_lens_out",
                                  "free_count_out", "token_offsets", "slots", "workspace"])
def test_plan_step_needs_its_buffers(name):
    assert plan(**{name: None}) == K.KVQ_ERR_INVALID_ARG


def test_integers_beyond_int32_are_refused_not_cut():
    with pytest.raises(K.KvqError):
        plan(max_tokens=(1 << 32) + 64)


# ------------------------------------------------------------------ prompt attention

def prompt(d=None, **kw):
    a = dict(q=FAKE, n_tokens=8, num_q_heads=16, k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE,
             page_table=FAKE, max_pages=4, seq_lens=FAKE, max_seq_len=256, token_offsets=FAKE, batch=2, causal=1,
             sm_scale=0.1, workspace=FAKE, workspace_bytes=1 << 40, out=FAKE, out_type=K.KVQ_OUT_F16)
    a.update(kw)
    return K.kvq_prompt_attn(d or desc(), *a.values(), stream=0, check=False)


@pytest.mark.parametrize("kw,code", [
    (dict(n_tokens=-1), K.KVQ_ERR_INVALID_ARG), (dict(num_q_heads=0), K.KVQ_ERR_INVALID_ARG),
    (dict(num_q_heads=18), K.KVQ_ERR_INVALID_ARG), (dict(num_q_heads=36), K.KVQ_ERR_UNSUPPORTED),
    (dict(batch=-1), K.KVQ_ERR_INVALID_ARG), (dict(batch=1025), K.KVQ_ERR_UNSUPPORTED),
    (dict(max_seq_len=-1), K.KVQ_ERR_INVALID_ARG), (dict(max_seq_len=(1 << 30) + 1), K.KVQ_ERR_UNSUPPORTED),
    (dict(max_pages=0), K.KVQ_ERR_INVALID_ARG), (dict(causal=2), K.KVQ_ERR_INVALID_ARG),
    (dict(out_type=2), K.KVQ_ERR_INVALID_ARG), (dict(sm_scale=float("nan")), K.KVQ_ERR_INVALID_ARG),
    (dict(sm_scale=float("inf")), K.KVQ_ERR_INVALID_ARG), (dict(sm_scale=1e300), K.KVQ_ERR_INVALID_ARG),
    (dict(workspace_bytes=255), K.KVQ_ERR_WORKSPACE), (dict(n_tokens=1 << 28), K.KVQ_ERR_UNSUPPORTED),
    (dict(page_table=None, max_pages=5), K.KVQ_ERR_INVALID_ARG),   # 2 * 5 pages of 8
    (dict(q=FAKE + 8), K.KVQ_ERR_INVALID_ARG), (dict(out=FAKE + 4), K.KVQ_ERR_INVALID_ARG),
    (dict(workspace=FAKE + 8), K.KVQ_ERR_INVALID_ARG), (dict(k_codes=FAKE + 2), K.KVQ_ERR_INVALID_ARG),
    (dict(n_tokens=0), K.KVQ_OK), (dict(batch=0), K.KVQ_OK)])
def test_prompt_refusals(kw, code):
    assert prompt(**kw) == code


@pytest.mark.parametrize("name", ["q", "k_codes", "k_scales", "v_codes", "v_scales", "seq_lens", "token_offsets",
                                  "workspace", "out"])
def test_prompt_needs_its_buffers(name):
    assert prompt(**{name: None}) == K.KVQ_ERR_INVALID_ARG


def test_prompt_refuses_bad_descriptors():
    assert prompt(desc(page_size=48)) == K.KVQ_ERR_UNSUPPORTED
    assert prompt(desc(head_dim=96)) == K.KVQ_ERR_UNSUPPORTED
    assert prompt(desc("lut4")) == K.KVQ_ERR_INVALID_ARG


# ------------------------------------------------------------------ shared prefixes

def prefix(d=None, **kw):
    a = dict(q=FAKE, batch=3, num_q_heads=16, k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE,
             prefix_table=FAKE, max_prefix_pages=4, prefix_lens=FAKE, max_prefix_len=256, group_offsets=FAKE,
             num_groups=2, page_table=FAKE, max_pages=2, seq_lens=FAKE, max_seq_len=128, sm_scale=0.1, workspace=FAKE,
             workspace_bytes=1 << 40, out=FAKE, out_type=K.KVQ_OUT_F32)
    a.update(kw)
    return K.kvq_prefix_attn(d or desc(), *a.values(), stream=0, check=False)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), K.KVQ_ERR_INVALID_ARG), (dict(batch=1025), K.KVQ_ERR_UNSUPPORTED),
    (dict(num_q_heads=36), K.KVQ_ERR_UNSUPPORTED), (dict(num_groups=0), K.KVQ_ERR_INVALID_ARG),
    (dict(num_groups=1025), K.KVQ_ERR_UNSUPPORTED), (dict(group_offsets=None), K.KVQ_ERR_INVALID_ARG),
    (dict(max_prefix_len=-1), K.KVQ_ERR_INVALID_ARG), (dict(max_seq_len=-1), K.KVQ_ERR_INVALID_ARG),
    (dict(max_seq_len=(1 << 30) + 1), K.KVQ_ERR_UNSUPPORTED), (dict(max_prefix_pages=0), K.KVQ_ERR_INVALID_ARG),
    (dict(prefix_table=None, max_prefix_pages=5), K.KVQ_ERR_INVALID_ARG),
    (dict(page_table=None, max_pages=3), K.KVQ_ERR_INVALID_ARG), (dict(out_type=7), K.KVQ_ERR_INVALID_ARG),
    (dict(sm_scale=float("-inf")), K.KVQ_ERR_INVALID_ARG), (dict(workspace_bytes=1024), K.KVQ_ERR_WORKSPACE),
    (dict(batch=0), K.KVQ_OK)])
def test_prefix_refusals(kw, code):
    assert prefix(**kw) == code


@pytest.mark.parametrize("name", ["q", "k_codes", "k_scales", "v_codes", "v_scales", "prefix_lens", "seq_lens",
                                  "workspace", "out"])
def test_prefix_needs_its_buffers(name):
    assert prefix(**{name: None}) == K.KVQ_ERR_INVALID_ARG


# ------------------------------------------------------------------ workspace sizes

def test_workspace_sizes():
    d = desc(num_kv_heads=8)
    # many row tiles: one split, written to the output directly
    assert K.kvq_prompt_workspace_size(d, 8192, 32, 1, 8192) == 256
    # few rows: 148 / 8 = 18 splits of whole 128-position tiles, 1024 positions each, so 16 of them;
    # a partial (o, m, l) of every split
    assert K.kvq_prompt_workspace_size(d, 4, 32, 1, 16384) == 256 + 4 * 32 * 16 * (128 + 2) * 4
    # lut4 rows are rotated back by the merge, so they always have partials
    lut = desc("lut4", num_kv_heads=8, codebook=FAKE, signs=FAKE)
    assert K.kvq_prompt_workspace_size(lut, 8192, 32, 1, 8192) == 256 + 8192 * 32 * (128 + 2) * 4
    assert K.kvq_prompt_workspace_size(d, -1, 32, 1, 10) == 0 and K.kvq_prompt_workspace_size(d, 1, 33, 1, 10) == 0
    assert K.kvq_prefix_workspace_size(d, 64, 32, 1, 32768, 1024) > 64 * 32 * 2 * 130 * 4
    assert K.kvq_prefix_workspace_size(d, 2000, 32, 1, 100, 100) == 0


# ------------------------------------------------------------------ the staging ring

class Barrier:
    """An mbarrier: a phase completes when its arrivals are in; a wait by parity passes when the
    phase of that parity is not the one under way."""

    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0, "more arrivals than the phase has"
        if self.left == 0:
            self.phase += 1
            self.left = self.count

    def passes(self, parity):
        return (self.phase & 1) != parity


def run_ring(stages, pieces, shared, rng):
    """A copier fills a ring of stages for two consumers in turn (pieces: whose each is), with
    copies landing in any order; returns whether each consumer only ever read its own piece."""
    full = [[Barrier(1) for _ in range(stages)] for _ in range(1 if shared else 2)]
    empty = [Barrier(1) for _ in range(stages)]
    stage_of = [i % stages for i in range(len(pieces))]
    holds = [None] * stages          # the piece whose copy has landed
    flight, copied = [], 0
    todo = [[i for i, who in enumerate(pieces) if who == w] for w in (0, 1)]
    bits = [[0] * stages, [0] * stages]
    while todo[0] or todo[1]:
        moves = []
        if copied < len(pieces):
            st = stage_of[copied]
            if copied < stages or empty[st].passes((copied // stages & 1) ^ 1):
                moves.append(("copy",))
        moves += [("land", i) for i in flight]
        for w in (0, 1):
            if todo[w]:
                i = todo[w][0]
                st = stage_of[i]
                parity = (i // stages & 1) if shared else bits[w][st]
                if full[0 if shared else w][st].passes(parity):
                    moves.append(("read", w, i, st))
        assert moves, "nobody can move"
        m = rng.choice(moves)
        if m[0] == "copy":
            flight.append(copied)
            copied += 1
        elif m[0] == "land":
            flight.remove(m[1])
            holds[stage_of[m[1]]] = m[1]
            full[0 if shared else pieces[m[1]]][stage_of[m[1]]].arrive()
        else:
            _, w, i, st = m
            if holds[st] != i:
                return False
            todo[w].pop(0)
            bits[w][st] ^= 1
            empty[st].arrive()
    return True


@pytest.mark.parametrize("stages", [3, 4, 6, 7])
def test_staging_ring_with_a_barrier_per_consumer(stages):
    # the rows kernel's ring: half tiles for two groups of warps, an odd one at the end
    for seed in range(300):
        rng = random.Random(seed)
        pieces = [0, 1] * rng.randint(1, 12)
        if rng.random() < 0.5:  # the last tile has one half: its K copy comes before the last V copies
            pieces = pieces[:-3] + [0] + pieces[-3:-1] + [0] if len(pieces) > 4 else pieces
        assert run_ring(stages, pieces, False, rng)


def test_staging_ring_with_one_barrier_per_stage_goes_wrong():
    # why each consumer has its own: with an odd number of stages a wait by parity can meet the
    # other consumer's phase
    assert not all(run_ring(3, [0, 1] * 6, True, random.Random(seed)) for seed in range(300))
