"""The latent calls' host side: every refusal before anything touches a GPU, and workspace sizes."""
import pytest

FAKE = 1 << 20  # 16-byte aligned dummy address; never dereferenced (rejected first)
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def kda():
    from kda_gated_delta_04_gb300 import build
    build.build()
    from kda_gated_delta_04_gb300 import kda as binding
    return binding


def append_args(**over):
    a = dict(latent=FAKE, latent_stride=576, k_pe=FAKE, k_pe_stride=576, norm_weight=FAKE, norm_eps=1e-6, cos_sin=FAKE,
             num_positions=10, positions=FAKE, q_pe=FAKE, q_token_stride=384, q_head_stride=192, q_pe_out=FAKE,
             out_token_stride=384, out_head_stride=192, latent_out=FAKE, latent_out_stride=512, k_pe_out=FAKE,
             k_pe_out_stride=64, num_tokens=4, num_heads=2, d_latent=512, d_pe=64, dtype=0, cache=FAKE, num_slots=64,
             slots=FAKE, device_errors=None, stream=None, flags=0)
    assert set(over) <= set(a)
    a.update(over)
    return a.values()


@pytest.mark.parametrize("over,expected", [
    (dict(latent=None), INVALID), (dict(k_pe=None), INVALID), (dict(cache=None), INVALID), (dict(slots=None), INVALID),
    (dict(latent=FAKE + 8), INVALID), (dict(q_pe=FAKE + 2), INVALID), (dict(cache=FAKE + 4), INVALID),
    (dict(cos_sin=FAKE + 4), INVALID), (dict(device_errors=FAKE + 1), INVALID),
    (dict(positions=None), INVALID), (dict(num_positions=0), INVALID),
    (dict(q_pe=None), INVALID), (dict(q_pe_out=None), INVALID), (dict(num_heads=0), INVALID),
    (dict(latent_stride=577), INVALID), (dict(q_head_stride=100), INVALID), (dict(out_token_stride=-8), INVALID),
    (dict(latent_out_stride=513), INVALID), (dict(k_pe_out_stride=3), INVALID), (dict(latent_stride=578, dtype=1), INVALID),
    (dict(norm_eps=-1.0), INVALID), (dict(norm_eps=float("nan")), INVALID), (dict(num_tokens=-1), INVALID),
    (dict(num_slots=-1), INVALID), (dict(dtype=2), INVALID), (dict(flags=2), INVALID), (dict(d_pe=0), INVALID),
    (dict(d_latent=256), UNSUPPORTED), (dict(d_pe=128), UNSUPPORTED),
    (dict(num_tokens=2 ** 31 - 1, num_heads=64), UNSUPPORTED), (dict(num_tokens=0, latent=None, slots=None), OK),
])
def test_append_refusals(kda, over, expected):
    assert kda.kda_latent_append(*append_args(**over)) == expected


def decode_args(**over):
    a = dict(q=FAKE, q_batch_stride=1152, q_head_stride=576, cache=FAKE, num_pages=8, page_size=64, page_table=FAKE,
             page_table_stride=4, max_pages=4, seq_lens=FAKE, batch=3, num_heads=2, d_latent=512, d_pe=64, dtype=0,
             scale=0.1, o=FAKE, lse=FAKE, workspace=FAKE, workspace_bytes=50331648, device_errors=None, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return a.values()


@pytest.mark.parametrize("over,expected", [
    (dict(q=None), INVALID), (dict(cache=None), INVALID), (dict(page_table=None), INVALID), (dict(seq_lens=None), INVALID),
    (dict(o=None), INVALID), (dict(workspace=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(cache=FAKE + 8), INVALID),
    (dict(page_table=FAKE + 2), INVALID), (dict(seq_lens=FAKE + 2), INVALID), (dict(o=FAKE + 8), INVALID),
    (dict(lse=FAKE + 2), INVALID), (dict(workspace=FAKE + 128), INVALID), (dict(workspace_bytes=100), INVALID),
    (dict(q_head_stride=577), INVALID), (dict(q_head_stride=0), INVALID), (dict(q_batch_stride=-8), INVALID), (dict(page_table_stride=-1), INVALID),
    (dict(batch=-1), INVALID), (dict(num_heads=0), INVALID), (dict(page_size=0), INVALID), (dict(num_pages=-1), INVALID),
    (dict(max_pages=-1), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(dtype=5), INVALID), (dict(d_latent=0), INVALID),
    (dict(page_size=12), UNSUPPORTED), (dict(d_latent=448), UNSUPPORTED), (dict(d_pe=32), UNSUPPORTED),
    (dict(num_pages=2 ** 26, page_size=64), UNSUPPORTED), (dict(batch=0, q=None, o=None, seq_lens=None), OK),
])
def test_decode_refusals(kda, over, expected):
    assert kda.kda_latent_decode(*decode_args(**over)) == expected


def prefill_args(**over):
    a = dict(q=FAKE, q_token_stride=384, q_head_stride=192, k_nope=FAKE, k_token_stride=512, k_head_stride=256, k_pe=FAKE,
             k_pe_stride=64, v=FAKE, v_token_stride=512, v_head_stride=256, cu_q=FAKE, cu_k=FAKE, num_seqs=2, q_tokens=10,
             k_tokens=20, num_heads=2, d_nope=128, d_pe=64, d_v=128, dtype=0, scale=0.1, o=FAKE, lse=FAKE,
             device_errors=None, stream=None, flags=0)
    assert set(over) <= set(a)
    a.update(over)
    return a.values()


@pytest.mark.parametrize("over,expected", [
    (dict(q=None), INVALID), (dict(k_nope=None), INVALID), (dict(k_pe=None), INVALID), (dict(v=None), INVALID),
    (dict(o=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(k_nope=FAKE + 8), INVALID), (dict(k_pe=FAKE + 8), INVALID),
    (dict(v=FAKE + 8), INVALID), (dict(o=FAKE + 8), INVALID), (dict(lse=FAKE + 2), INVALID), (dict(cu_q=FAKE + 2), INVALID),
    (dict(cu_k=FAKE + 2), INVALID), (dict(q_token_stride=100), INVALID), (dict(k_head_stride=-8), INVALID),
    (dict(k_pe_stride=65), INVALID), (dict(v_token_stride=3), INVALID),
    (dict(cu_q=None), INVALID),                       # cu_k alone
    (dict(cu_q=None, cu_k=None), INVALID),            # several sequences need offsets
    (dict(cu_k=None), INVALID),                       # as many keys as queries then
    (dict(num_seqs=0), INVALID), (dict(num_seqs=-1), INVALID), (dict(q_tokens=-1), INVALID), (dict(num_heads=0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(dtype=9), INVALID), (dict(flags=1), INVALID), (dict(d_v=0), INVALID),
    (dict(d_nope=64), UNSUPPORTED), (dict(d_v=64), UNSUPPORTED), (dict(d_pe=32), UNSUPPORTED),
    (dict(num_seqs=70000), UNSUPPORTED), (dict(q_tokens=2 ** 31), UNSUPPORTED),
    (dict(q_tokens=0, q=None, o=None), OK),
])
def test_prefill_refusals(kda, over, expected):
    assert kda.kda_latent_prefill(*prefill_args(**over)) == expected


def test_decode_workspace_size(kda):
    """Bounded whatever the heads; 0 for arguments the call refuses."""
    for dtype in (0, 1):
        for heads in (1, 16, 32, 33, 64, 100, 128, 1000):
            n = kda.kda_latent_decode_workspace_size(heads, dtype)
            assert 0 < n <= kda.KDA_LATENT_DECODE_WORKSPACE_MAX
    assert kda.kda_latent_decode_workspace_size(0, 0) == 0 and kda.kda_latent_decode_workspace_size(8, 2) == 0


def test_binding_refusals(kda):
    """Types, devices and shapes are refused in Python before an address is taken."""
    import torch
    x = torch.zeros(4, 576)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError):
        kda.latent_append(x[:, :512], x[:, 512:], torch.zeros(1, 8, 576), i)
    with pytest.raises(TypeError):
        kda.latent_append(x.half()[:, :512], x[:, 512:], torch.zeros(1, 8, 576), i)
    with pytest.raises(ValueError):
        kda.latent_append(x[:, :512], x[:, 512:], torch.zeros(1, 8, 576), i, positions=i)
    with pytest.raises(ValueError):
        kda.latent_append(x[:, :512], x[:, 512:], torch.zeros(8, 1, 576).transpose(0, 1)[:, ::2], i)
    with pytest.raises((TypeError, ValueError)):
        kda.latent_decode(torch.zeros(4, 2, 576), torch.zeros(1, 8, 576), torch.zeros(4, 1, dtype=torch.int32), i, 1.0)
    with pytest.raises(TypeError):
        kda.latent_prefill(torch.zeros(4, 2, 192), torch.zeros(4, 2, 128), torch.zeros(4, 64), torch.zeros(4, 2, 128), 1.0)
    with pytest.raises(ValueError):
        kda.latent_prefill(torch.zeros(4, 2, 192), torch.zeros(4, 2, 128), torch.zeros(4, 64), torch.zeros(4, 2, 128), 1.0,
                           cu_k=i)
