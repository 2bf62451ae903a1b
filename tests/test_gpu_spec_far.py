"""flint_verify_tree where offsets pass 2^31 elements."""
import pytest
import torch

from long_context_decode_flash_b200 import flint

pytestmark = pytest.mark.gpu


def test_rows_beyond_32_bit_offsets():
    """Five chains of three, rows 2^27 (target) and 3 2^26 (draft) values apart: the
    last rows lie 2.5e9 and 2.8e9 values on.  All accepted, the last request draws
    from its last target row; its last node rejected, from the residual of its last
    draft row."""
    B, N, V = 5, 3, 700
    g = torch.Generator().manual_seed(72)
    target = torch.softmax(torch.randn(B, N + 1, V, generator=g) * 2, -1).cuda()
    draft = torch.softmax(torch.randn(B, N, V, generator=g) * 2, -1).cuda()
    wide_t = torch.zeros(B * (N + 1) << 27, dtype=torch.float32, device="cuda").view(B, N + 1, 1 << 27)[..., :V]
    wide_d = torch.zeros(B * N * 3 << 26, dtype=torch.float32, device="cuda").view(B, N, 3 << 26)[..., :V]
    assert (wide_t[-1, -1].storage_offset() > 2 ** 31) and wide_d[-1, -1].storage_offset() > 2 ** 31
    wide_t.copy_(target)
    wide_d.copy_(draft)
    parent = torch.tensor([[-1, 0, 1]] * B, dtype=torch.int32, device="cuda")
    tokens = torch.stack([target[:, i].argmax(-1) for i in range(N)], 1).to(torch.int32)
    # the last node's token: offered more by the draft than the target gives
    tokens[-1, 2] = (target[-1, 2] - draft[-1, 2]).argmin()
    us = torch.rand(B, generator=g).cuda()
    seen = []
    for last in (0.0, 0.9999):
        ua = torch.zeros(B, N, device="cuda")
        ua[-1, 2] = last
        got = []
        for t, d in ((target, draft), (wide_t, wide_d)):
            path, n, token = torch.empty_like(tokens), torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
            flint.flint_verify_tree(t, d, tokens, parent, [N] * B, ua, us, path, n, token)
            got.append((path, n, token))
        for a, b in zip(*got):
            assert torch.equal(a, b)
        assert got[0][1].tolist() == [3, 3, 3, 3, 3 if last == 0.0 else 2]
        row = target[-1, 3].double() if last == 0.0 else (target[-1, 2].double() - draft[-1, 2].double()).clamp(min=0)
        c = row.cumsum(0)
        want = int((c > us[-1].double() * c[-1]).to(torch.uint8).argmax())
        seen.append(int(got[1][2][-1]) == want)
    assert all(seen)
