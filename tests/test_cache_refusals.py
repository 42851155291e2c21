"""Calls on the caches that are refused before anything is launched: the binding's own checks and the library's.  CPU only; where
the binding wants device tensors, host tensors stand in and the library's calls are replaced by a record of them."""
import pytest
import torch

from mtp_speculative_decode_gb300 import api


@pytest.fixture
def launches(monkeypatch):
    """The binding over host tensors; the names of the calls that would have been launched."""
    made = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: made.append(name) or 0

    monkeypatch.setattr(api, "lib", Lib)
    monkeypatch.setattr(api, "_stream", lambda stream: None)
    monkeypatch.setattr(api, "_need", lambda *a: None)
    return made


def rows(n, width, lead=()):
    dtype = {576: torch.bfloat16, 2304: torch.float32}.get(width, torch.uint8)
    return torch.zeros(*lead, n, 576 if width == 2304 else width, dtype=dtype)


def zeros(*shape, dtype=torch.int64):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("src,dst", [(656, 416), (416, 656)])
def test_write_back_between_packed_formats(launches, src, dst):
    """Both packed formats are bytes: rows of the one are no rows of the other (656-byte rows would run past a 416-byte pool)."""
    B, W = 2, 3
    acc = zeros(B, dtype=torch.int32)
    with pytest.raises(ValueError, match="rows"):
        api.kv_writeback(rows(W, src, (B,)), None, None, acc, rows(9, dst), None, None, zeros(B), zeros(B))
    with pytest.raises(ValueError, match="rows"):
        api.kv_writeback_slots(rows(W, src, (B,)), None, None, acc, rows(9, dst), None, None, zeros(B, W))
    assert launches == []


@pytest.mark.parametrize("width", [576, 2304, 656, 416])
def test_write_back_between_equal_formats(launches, width):
    B, W = 2, 3
    acc = zeros(B, dtype=torch.int32)
    api.kv_writeback(rows(W, width, (B,)), None, None, acc, rows(9, width), None, None, zeros(B), zeros(B))
    api.kv_writeback_slots(rows(W, width, (B,)), None, None, acc, rows(9, width), None, None, zeros(B, W))
    api.kv_move_accepted(rows(9, width), None, None, zeros(B, W), zeros(B, W, dtype=torch.int32), acc)
    assert launches == ["mtpsd_kv_writeback", "mtpsd_kv_writeback_slots", "mtpsd_kv_move_accepted"]


@pytest.mark.parametrize("bad", [torch.zeros(9, 512, dtype=torch.bfloat16), torch.zeros(9, 655, dtype=torch.uint8),
                                 torch.zeros(9, 576, dtype=torch.uint8), torch.zeros(9, 576, dtype=torch.float16)])
def test_rows_of_no_format(launches, bad):
    """The row's bytes come from its type and width: what is none of the formats has none."""
    B, W = 2, 3
    acc = zeros(B, dtype=torch.int32)
    with pytest.raises(ValueError, match="latent rows"):
        api.kv_move_accepted(bad, None, None, zeros(B, W), zeros(B, W, dtype=torch.int32), acc)
    with pytest.raises(ValueError, match="latent rows"):
        api.kv_writeback_slots(bad[:W].expand(B, W, -1), None, None, acc, bad, None, None, zeros(B, W))
    q = torch.zeros(1, 16, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="rows"):
        api.sparse_mla_decode(q, bad, zeros(1), zeros(2), zeros(1), zeros(1, 8, dtype=torch.int32), 1.0)
    assert launches == []
