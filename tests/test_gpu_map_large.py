"""The expert map at the largest number of slots it takes, 2^31 - 1 (17 GB of ids and rows)."""
from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import block_scaled_precision_bf16tofp4row_amd as mx  # noqa: E402


def test_most_slots():
    n, G = 2 ** 31 - 1, 2
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of free GPU memory")
    near = [np.arange(130), np.arange(n - 130, n)]
    near += [np.arange(s - 2, s + 3) for s in range(2 ** 21, n - 2 ** 10, 2 ** 21)]
    live = np.unique(np.concatenate(near))
    expert = live % 3                             # 2: of another rank
    ids = torch.full((n, 1), -1, dtype=torch.int32, device="cuda")
    at = torch.from_numpy(live).cuda()
    ids[at, 0] = torch.from_numpy(expert.astype(np.int32)).cuda()
    pos = torch.full((n, 1), -5, dtype=torch.int32, device="cuda")
    offs = torch.empty(G + 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(mx.mxfp4_expert_map_workspace(n, 1, G) // 4, dtype=torch.int32, device="cuda")
    mx.mxfp4_expert_map(ids, offs, pos, ws)
    first = int((expert == 0).sum())
    want = np.where(expert == 0, np.cumsum(expert == 0) - 1,
                    np.where(expert == 1, first + np.cumsum(expert == 1) - 1, -1))
    assert offs.tolist() == [0, first, first + int((expert == 1).sum())]
    assert np.array_equal(pos[at, 0].cpu().numpy(), want)
    none = sum(int((pos[a:a + 2 ** 28] == -1).sum()) for a in range(0, n, 2 ** 28))
    assert none == n - int((want >= 0).sum())
