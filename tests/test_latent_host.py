"""More of the latent calls' host side, without a GPU: calls whose outputs' rows overlap."""
import pytest
import torch

from test_latent_abi import FAKE, INVALID, append_args, kda  # noqa: F401 (a fixture)


@pytest.mark.parametrize("over", [
    dict(out_head_stride=0), dict(out_token_stride=0), dict(out_token_stride=0, out_head_stride=0),
    dict(out_head_stride=56), dict(out_head_stride=8),            # a row reaches into the next head's
    dict(out_token_stride=56, out_head_stride=1024),              # ... the next token's
    dict(out_token_stride=248), dict(out_token_stride=192),       # the heads of two tokens meet
    dict(out_token_stride=64, out_head_stride=248),               # heads outermost, the tokens of two heads meet
    dict(q_token_stride=0, q_head_stride=0, out_token_stride=384, out_head_stride=0),
    dict(num_heads=1, out_token_stride=0), dict(num_heads=1, out_token_stride=56),
    dict(num_tokens=1, out_head_stride=0), dict(num_tokens=1, out_head_stride=56),
    dict(latent_out_stride=0), dict(latent_out_stride=504), dict(k_pe_out_stride=0), dict(k_pe_out_stride=56),
    dict(out_token_stride=2 ** 37, out_head_stride=2 ** 38, num_tokens=2 ** 29),  # (products past 64 bits)
])
@pytest.mark.parametrize("dtype", [0, 1])
def test_append_refuses_outputs_that_overlap(kda, over, dtype):  # noqa: F811
    """Rows written by several warps: the result would hang on their order (in place, on how often a shared
    row had been rotated when it was read)."""
    assert kda.kda_latent_append(*append_args(**over, dtype=dtype)) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="passes every check, and the addresses are no one's")
@pytest.mark.parametrize("over", [
    dict(), dict(out_token_stride=64, out_head_stride=256), dict(out_token_stride=128, out_head_stride=64),
    dict(out_token_stride=256, out_head_stride=192), dict(num_tokens=1, out_token_stride=0, latent_out_stride=0, k_pe_out_stride=0),
    dict(num_heads=1, out_head_stride=0), dict(num_tokens=1, num_heads=1, out_token_stride=0, out_head_stride=0),
    dict(q_token_stride=0, q_head_stride=0), dict(latent_stride=0, k_pe_stride=0),  # inputs may be shared
    dict(latent_out=None, latent_out_stride=0), dict(k_pe_out=None, k_pe_out_stride=0),
    dict(q_pe=None, q_pe_out=None, out_token_stride=0, out_head_stride=0),
    dict(latent_out_stride=512, k_pe_out_stride=64),
])
def test_append_takes_outputs_that_do_not(kda, over):  # noqa: F811
    """Past the checks of the arguments the entry point finds that there is no device."""
    assert kda.kda_latent_append(*append_args(**over)) == kda.KDA_ERR_CUDA
