"""Dense paged decode of rows whose logits are all -inf over value rows that are not finite: such a row is
empty, out = 0 and lse = -inf, whatever its values hold (0 times them is not 0)."""
import pytest
import torch

import sparse_decode_attention_quest_gb300 as se

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_errors(se_lib, cuda_device):
    se.se_read_device_error(clear=True)
    yield
    assert se.se_read_device_error(clear=True) == 0


@pytest.mark.parametrize("wide", [False, True])  # of wide tables the joins run in a kernel of their own
@pytest.mark.parametrize("lens", [[40], [9000], [300] * 160, [5000, 3, 17, 2000]])
@pytest.mark.parametrize("Hq,H,D", [(8, 2, 128), (4, 1, 64), (8, 8, 128), (40, 1, 256), (32, 1, 64), (16, 1, 576),
                                    (64, 1, 576)])
def test_rows_without_a_finite_logit(cuda_device, Hq, H, D, lens, wide):
    dev, g = cuda_device, torch.Generator().manual_seed(1)
    Dv = 512 if D == 576 else D
    n = [-(-x // 16) for x in lens]
    table = torch.zeros(len(lens), 4096 if wide else max(n), dtype=torch.int32)
    for b, m in enumerate(n):
        table[b, :m] = torch.arange(m) + sum(n[:b])
    k = torch.randn(sum(n), H, 16, D, generator=g).to(torch.bfloat16)
    v = None if D == 576 else torch.randn(sum(n), H, 16, D, generator=g).to(torch.bfloat16)
    q = torch.randn(len(lens), Hq, D, generator=g).to(torch.bfloat16)
    # Every other request: keys of -inf against queries of 1, in a value dim of the latent cache.
    q[..., 5] = 1
    for b in range(0, len(lens), 2):
        pages = table[b, :n[b]].long()
        k[pages, ..., 5] = -float("inf")
        if v is not None:
            v[pages, ..., 7] = float("nan")
            v[pages, ..., 9] = float("inf")
    out = torch.full((len(lens), Hq, Dv), 77.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((len(lens), Hq), 77.0, device=dev)
    ws = torch.zeros(se.se_paged_decode_workspace_size(len(lens), Hq, H, D, Dv), dtype=torch.uint8, device=dev)
    dk, dv = k.to(dev), None if v is None else v.to(dev)
    se.se_paged_decode(se.paged_kv(dk, dv, None, Dv), q.to(dev), table.to(dev),
                       torch.tensor(lens, dtype=torch.int32, device=dev), D ** -0.5, out, lse, ws)
    torch.cuda.synchronize()
    assert bool((out[::2] == 0).all()) and bool(torch.isneginf(lse[::2]).all())
    assert bool(torch.isfinite(out[1::2]).all()) and bool(torch.isfinite(lse[1::2]).all())
