"""The norm and its backward in flight on two streams: every output bit for bit as if alone."""
import pytest
import torch

from fp8_ref import F8, groups

pytestmark = pytest.mark.gpu


def case(seed, rows, dim, dtype):
    import hybrid_masked_attention_b200 as M
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, dy, dres, w = rnd(rows, dim).to(dtype), rnd(rows, dim).to(dtype), rnd(rows, dim).to(dtype), 1 + 0.2 * rnd(dim)
    out = {"q": torch.empty(rows, dim, dtype=F8, device="cuda"), "s": torch.empty(rows, groups(dim), device="cuda"),
           "rstd": torch.empty(rows, device="cuda"), "dx": torch.empty_like(x), "dw": torch.empty(dim, device="cuda")}
    ws = torch.empty(M.rmsnorm_bwd_workspace_bytes(rows, dim), dtype=torch.uint8, device="cuda")

    def call(stream=None):
        M.add_rmsnorm_fp8(x, None, w, None, out["q"], out["s"], out["rstd"], stream=stream)
        M.rmsnorm_bwd(x, w, out["rstd"], dy, dres, out["dx"], out["dw"], ws, stream=stream)

    return call, out


@pytest.mark.parametrize("shapes", [((3000, 512), (2500, 768)), ((700, 4096), (300, 9000)), ((1, 512), (20000, 96))], ids=str)
def test_norms_and_backwards_on_two_streams(shapes, cuda_ok):
    cases = [case(11 + i, *s, t) for i, (s, t) in enumerate((s, t) for s in shapes for t in (torch.float32, torch.bfloat16))]
    want = []
    for call, out in cases:
        call()
        want.append({k: t.clone() for k, t in out.items()})
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(8):
        for _, out in cases:
            for t in out.values():
                t.view(torch.uint8).fill_(0xFF)
        torch.cuda.synchronize()
        for i, (call, _) in enumerate(cases):
            call(streams[(i + rep) % 2])
        torch.cuda.synchronize()
        for (_, out), w in zip(cases, want):
            for k in w:
                assert torch.equal(out[k].view(torch.uint8), w[k].view(torch.uint8)), k
