"""Host-only checks of the serving calls at the ends of their ranges (nothing is launched)."""
import pytest

import quantized_kv_cache_split_b200 as K

FAKE = 1 << 20  # aligned dummy device pointer


def desc(fmt="q8_0", head_dim=128, num_kv_heads=4, page_size=64, num_pages=8):
    args = (FAKE, FAKE) if fmt == "lut4" else (None, None)
    return K.make_desc(fmt, head_dim, num_kv_heads, page_size, num_pages, *args)


# ------------------------------------------------------------------ workspaces of the longest sequences

def partials(rows, splits, head_dim):
    return rows * splits * (head_dim + 2) * 4


@pytest.mark.parametrize("batch", [1, 37, 1024])
@pytest.mark.parametrize("hkv", [1, 4, 6, 8, 12, 16, 64])
def test_prefix_workspace_holds_a_partial_of_both_parts(batch, hkv):
    rows = batch * hkv * 4
    for fmt in ("q8_0", "lut4"):
        for prefix in (0, 4096, 1 << 29):
            for own in (1, 1000, 1 << 20, (1 << 29) - 1, 1 << 29):
                size = K.kvq_prefix_workspace_size(desc(fmt, num_kv_heads=hkv), batch, hkv * 4, 1, prefix, own)
                # one (o, m, l) per row of the prefix and one of the request's own positions at the
                # least, and no more splits than there are SMs, and warps on them
                assert size >= 256 + 2 * partials(rows, 1, 128), (fmt, prefix, own)
                assert size <= 512 + partials(rows, 148 + 148 * 12 // (batch * hkv) + 1, 128), (fmt, prefix, own)


# ------------------------------------------------------------------ a flag word outside the workspace

def test_flag_words_must_be_aligned():
    for flags in (FAKE + 1, FAKE + 2):
        assert K.kvq_prompt_attn(desc(), FAKE, 8, 16, FAKE, FAKE, FAKE, FAKE, FAKE, 4, FAKE, 256, FAKE, 2, 1, 0.1, FAKE,
                                 1 << 40, FAKE, stream=0, check=False, flags=flags) == K.KVQ_ERR_INVALID_ARG
        assert K.kvq_prefix_attn(desc(), FAKE, 8, 16, FAKE, FAKE, FAKE, FAKE, FAKE, 4, FAKE, 256, FAKE, 2, FAKE, 2, FAKE,
                                 128, 0.1, FAKE, 1 << 40, FAKE, stream=0, check=False, flags=flags) == K.KVQ_ERR_INVALID_ARG


# ------------------------------------------------------------------ calls without work

def test_calls_without_work_need_no_buffers():
    # the address of a tensor without elements is 0
    none = [None] * 4
    assert K.kvq_plan_step(0, 64, 8, 4, 16, None, None, FAKE, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, FAKE, 256, stream=0,
                           check=False) == K.KVQ_OK
    for n, batch, q, lens in ((0, 2, None, FAKE), (8, 0, FAKE, None), (0, 0, None, None)):
        assert K.kvq_prompt_attn(desc(), q, n, 16, FAKE, FAKE, FAKE, FAKE, None, 4, lens, 256, FAKE, batch, 1, 0.1, FAKE,
                                 256, q, stream=0, check=False) == K.KVQ_OK
    assert K.kvq_prefix_attn(desc(), None, 0, 16, *none, None, 4, None, 256, None, 1, None, 4, None, 128, 0.1, None, 0, None,
                             stream=0, check=False) == K.KVQ_OK
    # what is wrong about them is still refused
    assert K.kvq_prompt_attn(desc(), None, 0, 18, *none, None, 4, None, 256, None, 0, 1, 0.1, None, 0, None, stream=0,
                             check=False) == K.KVQ_ERR_INVALID_ARG


def test_packed_call_refuses_what_it_does_not_know():
    assert K.kvq_packed_call(3, b"\0" * 256, check=False) == K.KVQ_ERR_INVALID_ARG
    assert K.kvq_packed_call(1, None, check=False) == K.KVQ_ERR_INVALID_ARG
    assert K.kvq_packed_call(1, b"\0" * 256, check=False) == K.KVQ_ERR_INVALID_ARG   # no descriptor
    with pytest.raises(K.KvqError):
        K.kvq_packed_call(-1, b"\0" * 256)
