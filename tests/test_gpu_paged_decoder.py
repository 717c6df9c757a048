"""The end-to-end loop over a paged cache: prefill, greedy decoding, the
consensus loop and filtered sampling on the random-init decoder, with and
without a prompt that all sequences share.

In FP32 the paged attention is row-invariant, so the consensus loop emits the
greedy tokens exactly, as over the dense cache."""
import numpy as np
import pytest
import torch

import block_attention_b200 as ba
from block_attention_b200 import synth
from block_attention_b200.decoder import AR_VIEW, DecodeState, PagedState, TinyDecoder
from gpu_util import to_host

pytestmark = pytest.mark.gpu

V, D_MODEL, LAYERS, HQ, HKV, HD, FFN = 1000, 128, 2, 4, 2, 64, 256


@pytest.fixture(scope="module")
def weights():
    return synth.decoder_weights(V, D_MODEL, LAYERS, HQ, HKV, HD, FFN, seed=77, std=0.05)


def model(weights, dtype):
    return TinyDecoder(weights, HQ, HKV, HD, dtype=dtype)


def prompts(shared=0, seed=0):
    g = np.random.default_rng(seed)
    head = g.integers(0, V - 1, shared).tolist()
    return [head + g.integers(0, V - 1, n).tolist() for n in (1, 40, 17, 70, 33)]


@pytest.mark.parametrize("shared,page_size", [(0, 16), (0, 64), (50, 16), (64, 64)])
def test_fp32_consensus_over_pages_is_greedy(weights, shared, page_size):
    m = model(weights, torch.float32)
    p = prompts(shared)
    kw = dict(page_size=page_size, shared=shared)
    ref = m.greedy(p, 40, cap=256, **kw)
    got, stats = m.consensus(p, 40, cap=256, **kw)
    np.testing.assert_array_equal(got, ref)
    assert stats["rounds"] > 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shared", [0, 50])
def test_prefill_over_pages_matches_the_dense_cache(weights, dtype, shared):
    """K/V of the first layer do not pass through attention: equal bits; the
    next block's logits agree to the forward pass's rounding."""
    m = model(weights, dtype)
    p = prompts(shared, seed=1)
    dense, first_d, _ = m.prefill(p, 192)
    paged, first_p, _ = m.prefill(p, 192, page_size=16, shared=shared)
    assert isinstance(dense, DecodeState) and isinstance(paged, PagedState)
    assert paged.prefix == shared // 16 * 16
    assert torch.equal(dense.ctx_lens, paged.ctx_lens)
    flat = paged.k[:, paged.table.long()].permute(0, 1, 3, 2, 4, 5).reshape(
        m.L, paged.B, m.Hkv, -1, m.hd)
    for b, n in enumerate(dense.ctx_lens.tolist()):
        assert torch.equal(flat[0, b, :, :n], dense.k[0, b, :, :n])
    tok = torch.from_numpy(np.random.default_rng(2).integers(0, V - 1, (5, 4)).astype(
        np.int32)).cuda()
    a = to_host(m.forward(dense, tok, AR_VIEW)[0])
    b = to_host(m.forward(paged, tok, AR_VIEW)[0])
    # the bounds of the decoder's own forward tests (1e-4 FP32, 8e-2 BF16 of a row's largest logit)
    tol = 1e-4 if dtype == torch.float32 else 8e-2
    assert (np.abs(a - b).max(1) <= 2 * tol * np.abs(a).max(1)).all()


def test_filtered_sampling_decodes_from_the_kept_tokens(weights):
    m = model(weights, torch.float32)
    p = prompts(20, seed=3)
    greedy = m.greedy(p, 24, cap=192)
    # top_k 1 and temperature 0 are greedy whatever the uniforms; pages change nothing
    for kw in (dict(temperature=0.7, top_k=1), dict(temperature=0.0, top_p=0.9)):
        np.testing.assert_array_equal(m.sample_ar(p, 24, seed=5, cap=192, **kw), greedy)
    paged = m.sample_ar(p, 24, 0.0, seed=5, cap=192, top_k=3, page_size=32, shared=20)
    np.testing.assert_array_equal(paged, m.greedy(p, 24, cap=192, page_size=32, shared=20))
    a = m.sample_ar(p, 24, 0.9, seed=5, cap=192, top_k=30, top_p=0.95, min_p=0.01)
    b = m.sample_ar(p, 24, 0.9, seed=5, cap=192, top_k=30, top_p=0.95, min_p=0.01)
    np.testing.assert_array_equal(a, b)
    assert ((a >= 0) & (a < V)).all() and (a[:, 1:] != greedy[:, 1:]).any()


def test_shared_prompt_is_checked(weights):
    m = model(weights, torch.float32)
    with pytest.raises(ValueError):
        m.prefill([[1, 2, 3], [1, 9, 3]], 64, page_size=16, shared=2)
    with pytest.raises(ValueError):
        m.prefill([[1, 2], [1, 2, 3]], 64, page_size=16, shared=2)
    with pytest.raises(ValueError):
        m.prefill([[1, 2, 3]], 64, shared=2)
