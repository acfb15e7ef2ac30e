"""The launches that batches of different sizes take in usaf_gate_topk: on both sides of each border, the tables
of every chunk, and longer batches of few experts."""
import pytest

from test_gpu_gate import check, data, device, pytestmark  # noqa: F401


@pytest.mark.parametrize("T,E,k", [
    (4096, 8, 2), (4097, 8, 2),           # 128 chunks, 129
    (4096, 128, 2), (4065, 130, 2),       # 16,384 words of masks, 128 * 130
    (2048, 256, 2), (2049, 256, 2),       # 64 chunks of 256, 65
    (512, 1024, 4), (513, 1024, 4),
    (20000, 4, 1)])
def test_tables_with_and_without_the_scan(T, E, k):
    l, b = data(T, E, T % 97)
    check(device(), l, k, dict(score="sigmoid"), b)
