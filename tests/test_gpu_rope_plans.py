"""kvq_norm_rope takes more tokens per CTA on longer prompts: the same bits as from short calls, on
both sides of every change of plan, for head layouts of which one to sixteen tokens fit a CTA."""
import pytest
import torch

from layer_wise_mixed_b200 import kvq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hkv,G,D", [(2, 6, 128), (4, 7, 64), (1, 4, 128), (1, 1, 64)])
@pytest.mark.parametrize("tokens", [3551, 3552, 3553, 7104, 7111, 14207, 14208, 14219])
def test_same_bits_in_short_calls(tokens, Hkv, G, D):
    W = (Hkv * G + 2 * Hkv) * D
    cache = kvq.Cache(1, 1, Hkv, Hkv * G, D, 8, [(4, 4)])
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn((1, tokens, W), generator=g, device="cuda").to(torch.bfloat16)
    w = 1 + 0.3 * torch.randn(D, generator=g, device="cuda")
    rope = kvq.Rope(D // 2, (1e4 ** (-torch.arange(0, D // 2, 2, device="cuda") / (D // 2))).float(), w, w, 1e-6, True)
    q, K, V = cache.norm_rope(0, x, rope)
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")[None]
    for a in list(range(0, tokens, 887)) + [tokens - 1]:
        b = min(a + 887, tokens)
        qs, Ks, Vs = cache.norm_rope(0, x[:, a:b], rope, pos[:, a:b].contiguous())
        assert torch.equal(q[:, a:b], qs) and torch.equal(K[:, :, a:b], Ks) and torch.equal(V[:, :, a:b], Vs), (a, b)
