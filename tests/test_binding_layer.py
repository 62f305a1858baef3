"""The binding's structs are filled from tensors whose shapes and types are checked (no GPU needed)."""
import pytest
import torch

import weight_only_int4_tma_gb300 as w4


def _config(table, rot_dim=64):
    return w4.rope_config(8, 2, 64, w4.W4A16_BF16, table, rot_dim)


def test_rope_config_takes_its_table():
    table = torch.empty(100, 64)
    cfg = _config(table)
    assert cfg.table == table.data_ptr() and cfg.table_len == 100 and cfg.rot_dim == 64
    assert _config(None, 0).table_len == 0x7FFFFFFF
    assert _config(table[:50]).table_len == 50
    assert _config(table.view(100, 2, 32)).table_len == 100  # cosines and sines apart


@pytest.mark.parametrize("table", [None, torch.empty(100, 32), torch.empty(100, 128), torch.empty(6400),
                                   torch.empty(100, 2, 64), torch.empty(100, 64, dtype=torch.float64),
                                   torch.empty(100, 64, dtype=torch.bfloat16), torch.empty(100, 128)[:, :64],
                                   torch.empty(64, 100).t()], ids=lambda t: t is None or f"{tuple(t.shape)}{t.stride()}{t.dtype}")
def test_rope_config_refuses_other_tables(table):
    """Read as float32 [positions][rot_dim], a table of another shape or type would be read past its end."""
    with pytest.raises(w4.W4A16Error):
        _config(table)
