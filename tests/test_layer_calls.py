"""What the Python entry points of a decoder layer's operators hand to the C ABI (no GPU)."""
import pytest
import torch

import quantized_gemm_amd as qg


class Seen:
    """Stands for the library: keeps the arguments of the calls."""

    def __init__(self):
        self.args = None

    def qg_attention(self, *args):
        self.args = args
        return 0


@pytest.fixture
def seen(monkeypatch):
    s = Seen()
    monkeypatch.setattr(qg, "lib", lambda: s)
    return s


def _attention(table, batch, max_len=64, page=16):
    d = qg.make_kv_desc(qg.O_BF16, 1, 64, page, 9)
    q = torch.zeros((max(batch, 1), 64), dtype=torch.bfloat16)
    qg.attention(d, q, 1, q, table, torch.zeros(batch, dtype=torch.int32), batch, max_len, 1.0, q, tokens=batch, stream=0)


@pytest.mark.parametrize("first,pages", [(0, 4), (3, 4), (0, 11), (5, 6)])
def test_attention_takes_the_rows_of_a_wider_table(seen, first, pages):
    wide = torch.arange(55, dtype=torch.int32).reshape(5, 11)
    table = wide[1:4, first:first + pages]
    _attention(table, 3)
    assert seen.args[5] == table.data_ptr() and seen.args[6] == 11
    _attention(wide[::2, first:first + pages], 3)
    assert seen.args[6] == 22


def test_attention_takes_tables_of_one_row_and_none(seen):
    row = torch.zeros(20, dtype=torch.int32)
    for t in (row[:4], row[:4][None], row.reshape(2, 10)[:1, :4]):
        _attention(t, 1)
        assert seen.args[5] == t.data_ptr() and seen.args[6] >= 4
    _attention(row.reshape(5, 1, 4), 5)
    assert seen.args[6] == 4
    _attention(None, 1, max_len=0)
    assert seen.args[5] is None and seen.args[6] == 0


def test_attention_refuses_tables_it_cannot_read(seen):
    wide = torch.zeros((3, 20), dtype=torch.int32)
    for t, max_len in ((wide[:, ::2], 64), (wide.t(), 16), (wide[:, :4], 65), (wide.reshape(3, 4, 5)[:, :, :4], 64)):
        with pytest.raises(qg.QGError):
            _attention(t, 3, max_len)
    assert seen.args is None
