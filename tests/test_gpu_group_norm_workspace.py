"""The group norm's gradients in a workspace of the size that the library names, between
guards: all of it may be used and nothing beside it."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,groups,width", [(700, 3, 64), (1, 1, 7), (3000, 24, 75), (5000, 1, 1536), (9, 2, 12_001), (40, 1, 20_001)])
def test_named_size(rows, groups, width, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import spectral_optimizer_ssm_amd as mu
    gen = torch.Generator(device="cuda").manual_seed(width)
    x, z, dy = (torch.randn(rows, groups * width, generator=gen, device="cuda").to(dtype) for _ in range(3))
    w = torch.rand(groups * width, generator=gen, device="cuda")
    need = mu.muon_group_norm_backward_workspace_size(x, groups)
    buf = torch.full((need + 512,), 165, dtype=torch.uint8, device="cuda")
    for kw in (dict(gate=z), dict(gate=z, gate_first=False), dict(), dict(activation="none")):
        _, mean, rstd = mu.muon_group_norm(x, groups, w, w, center=True, **kw)
        a = (dy, x, groups, w, w, mean, rstd)
        want = mu.muon_group_norm_backward(*a, center=True, **kw)
        got = mu.muon_group_norm_backward(*a, center=True, workspace=buf[256:-256], **kw)
        assert all(g is v or torch.equal(g, v) for g, v in zip(got, want))
        assert (buf[:256] == 165).all() and (buf[-256:] == 165).all()
