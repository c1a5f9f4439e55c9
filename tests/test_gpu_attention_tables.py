"""kv_cache_attention over page tables that have no column to spare, or one or two, at lengths where a sequence begins to be
split into parts: every row is written, whatever the output held."""
import math

import pytest
import torch

from nvfp4_block_scaled_moe_amd import ops
from tests.attention_util import BF, Case, check

pytestmark = pytest.mark.gpu


def _tight(c, cols, window=0):
    """The case's attention through a table of ``cols`` columns, into an output of NaN."""
    assert max(c.total) <= cols * c.page
    table = torch.full((len(c.new), cols), -1, dtype=torch.int32)
    used = -(-max(c.total) // c.page)
    table[:, :used] = c.table[:, :used]
    batch = ops.CacheBatch(table.cuda(), c.batch.lengths, c.batch.starts)
    got = ops.kv_cache_attention(c.q.cuda(), c.cache, batch, window=window, out=torch.full(c.q.shape, math.nan, dtype=BF, device="cuda"))
    check(got, *c.attention(window=window), f"{c.total} tokens in {cols} columns of {c.page}")


# (page, columns, lengths): blocks of 32 keys (bf16) or 64 (E4M3) are split from 24 on, tables end at, before and behind one's end
FEW = {False: [(16, 46, (721, 736)), (16, 47, (736, 737, 752)), (16, 48, (737, 753, 768)), (32, 23, (736,)), (32, 24, (737, 768)),
               (64, 12, (737, 768))],
       True: [(16, 92, (1457, 1472)), (16, 93, (1472, 1473, 1488)), (16, 94, (1473, 1504)), (16, 95, (1473, 1505, 1520)),
              (16, 96, (1473, 1521, 1536)), (32, 46, (1472,)), (32, 47, (1472, 1473, 1504)), (32, 48, (1473, 1536)), (64, 24, (1473, 1536))]}
# of 64 keys, from 12 on
MANY = [(16, 44, (689, 704)), (16, 45, (704, 705, 720)), (16, 46, (705, 736)), (16, 47, (705, 737, 752)), (16, 48, (705, 753, 768)),
        (32, 22, (704,)), (32, 23, (704, 705, 736)), (32, 24, (705, 768)), (64, 12, (705, 768))]
FLAT = lambda table: [(page, cols, n) for page, cols, lengths in table for n in lengths]  # noqa: E731


@pytest.mark.parametrize("fp8,page,cols,n", [(f, *x) for f in FEW for x in FLAT(FEW[f])])
def test_single_tokens(fp8, page, cols, n):
    c = Case([1], [n - 1], 8, 1, 64, page, fp8=fp8, seed=n)
    assert c.rows() <= 16
    _tight(c, cols)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page,cols,n", FLAT(MANY))
def test_many_rows(page, cols, n, fp8):
    _tight(Case([40], [n - 40], 8, 1, 64, page, fp8=fp8, seed=n), cols)


@pytest.mark.parametrize("D", [32, 96, 128, 160, 256])
@pytest.mark.parametrize("fp8,cols", [(False, 47), (True, 95)])
def test_head_sizes(D, fp8, cols):
    _tight(Case([1], [16 * cols - 9], 4, 2, D, 16, fp8=fp8, seed=D), cols)
    _tight(Case([20], [47 * 16 - 29], 4, 2, D, 16, fp8=fp8, seed=D + 1), 47)


@pytest.mark.parametrize("fp8,cols", [(False, 47), (True, 95)])
def test_a_batch_whose_longest_sequence_fills_the_table(fp8, cols):
    n = 16 * cols
    _tight(Case([1] * 5, [n - 1, 3, n - 16, 200, n - 20], 16, 2, 64, 16, fp8=fp8, seed=1), cols)
    _tight(Case([1, 90, 2], [700, 640, 5], 8, 2, 64, 16, fp8=fp8, seed=2), 47)


@pytest.mark.parametrize("new", [1, 40])
def test_a_window_nearly_as_long_as_the_table(new):
    _tight(Case([new], [752 - new], 8, 1, 64, 16, seed=3), 47, window=745)


def test_a_sequence_that_grows_to_its_table_end():
    """One request decoding, its table as wide as it ever gets, its length past the last steps."""
    c = Case([1], [751], 4, 1, 32, 16, seed=4)
    table, q = c.batch.page_table[:, :47].contiguous(), c.q.cuda()
    for n in range(730, 753):
        batch = ops.CacheBatch(table, torch.tensor([n], dtype=torch.int32, device="cuda"), c.batch.starts)
        wide = ops.CacheBatch(c.batch.page_table, batch.lengths, c.batch.starts)
        out = torch.full_like(q, math.nan)
        assert torch.equal(ops.kv_cache_attention(q, c.cache, batch, out=out), ops.kv_cache_attention(q, c.cache, wide)), n
