"""The binding takes a call's scale by its value: a tensor that was changed in place since the last call counts as it is
now, and whatever float() takes is taken."""

import numpy as np
import pytest

import gated_deltanet_scan_gb300 as gdr
from tests import gpu_util as gu


def dims_of(torch):
    return (lambda scale: gdr._attn_dims(16, 4, 256, torch.bfloat16, scale),
            lambda scale: gdr._tree_dims(16, 32, 128, 128, torch.bfloat16, torch.float32, scale, 0))


def test_a_scale_changed_in_place_counts_as_it_is_now():
    torch = pytest.importorskip("torch")
    for dims in dims_of(torch):
        for scale in (torch.tensor(0.5), torch.nn.Parameter(torch.tensor([0.5])), np.array(0.5), np.array([0.5])[0:1].reshape(())):
            assert dims(scale).scale == 0.5
            with torch.no_grad():
                scale.fill(0.25) if isinstance(scale, np.ndarray) else scale.fill_(0.25)
            assert dims(scale).scale == 0.25
            assert dims(0.5).scale == 0.5


def test_scales_of_every_kind():
    torch = pytest.importorskip("torch")
    for dims in dims_of(torch):
        for scale in (2, True, np.float32(0.3), np.float64(0.3), np.array(0.3), torch.tensor(0.3), torch.tensor(3)):
            assert dims(scale).scale == np.float32(float(scale))
        for scale in (torch.tensor([0.5, 0.5]), 1j, [0.5]):
            with pytest.raises((TypeError, ValueError, RuntimeError)):
                dims(scale)
    assert gdr._attn_dims(16, 4, 256, torch.bfloat16, None).scale == 0.0625


@pytest.mark.gpu
def test_calls_go_by_the_scale_as_it_is():
    torch = gu.require_gpu()
    gen = torch.Generator(device="cuda").manual_seed(1)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    n, n_tok, h, d = 2, 3, 2, 64
    q, k, v = randn(n * n_tok, h, d), randn(n * n_tok, h, d), randn(n * n_tok, h, d)
    cu = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    kc, vc = randn(4, 16, h, d), randn(4, 16, h, d)
    table = torch.tensor([[2, 0], [1, 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([30, 20], dtype=torch.int32, device="cuda")
    parents = torch.tensor([[-1, 0, 0]] * n, dtype=torch.int32, device="cuda")
    g, beta = -randn(n * n_tok, h).float().abs(), randn(n * n_tok, h).float().sigmoid()
    state = randn(n, h, d, d, dtype=torch.float32)
    calls = (
        lambda o, s: gdr.gdr_attn_prefill(q, k, v, o, cu, scale=s),
        lambda o, s: gdr.gdr_attn_decode(q, kc, vc, table, lens, o, n_tok, scale=s),
        lambda o, s: gdr.gdr_attn_decode_tree(q, kc, vc, table, lens, o, parents, scale=s),
        lambda o, s: gdr.gdr_verify_tree(q, k, v, g, beta, state, o, parents, scale=s),
    )
    for call in calls:
        want, got = ([torch.empty_like(q) for _ in range(2)] for _ in range(2))
        scale = torch.tensor(0.5)
        for i, x in enumerate((0.5, 0.125)):
            call(want[i], x)
            scale.fill_(x)
            call(got[i], scale)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)) and not torch.equal(*got)
