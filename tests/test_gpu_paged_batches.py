"""paged_attention over batches of more tiles than compute units with one sequence far longer than the
others, and over pages of any size (MI355X), against the float64 oracle."""
import pytest
import torch

from block_helpers import DEV
from test_gpu_paged_attention import check, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Q", [1, 3, 70])
@pytest.mark.parametrize("at", [0, 17, 39])
def test_one_long_sequence_among_many(at, Q):
    """320 key heads of sequences: the long one in the first round, in the middle, and in the cut tiles."""
    lens = [20 + 7 * b for b in range(40)]
    lens[at] = 6000
    q, kc, vc, table, l = inputs(40, Q, 16 if Q == 1 else 8, 8, 64, 16, lens, "bf16")
    check(q, kc, vc, table, l, f"{at}")
    lens[at] = 2
    check(q, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device=DEV), "none long, a wide table")


@pytest.mark.parametrize("page", [4112, 65536 + 16, 2**20 - 16, 2**20])
def test_large_pages(page):
    """Few keys of large pages, on both sides of a page's end."""
    for Q, dtype in ((1, "bf16"), (40, "f16")):
        n = page + 70
        g = torch.Generator().manual_seed(page % 1000)
        kc, vc = (torch.full((3, page, 1, 8), float("nan"), device=DEV) for _ in range(2))
        table = torch.tensor([[2, 0]], dtype=torch.int32, device=DEV)
        # the second page's keys alone have a share: the first page's are left out (no page)
        table[0, 0] = -1
        for c in (kc, vc):
            c[0, :70] = torch.randn(70, 1, 8, generator=g).to(DEV)
        q = torch.randn(1, Q, 4, 8, generator=g).to(DEV)
        q, kc, vc = (t.bfloat16() if dtype == "bf16" else t.half() for t in (q, kc, vc))
        check(q, kc, vc, table, torch.tensor([n], dtype=torch.int32, device=DEV), f"page {page} {Q}")
