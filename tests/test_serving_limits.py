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
