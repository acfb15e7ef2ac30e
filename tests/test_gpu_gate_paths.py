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


@pytest.mark.parametrize("E,G,Gk", [(65, 5, 2), (96, 8, 3), (96, 1, 1), (93, 3, 2), (129, 3, 1), (160, 32, 9), (161, 7, 2),
                                    (192, 8, 3), (186, 31, 12), (257, 1, 1), (264, 8, 5), (384, 8, 3), (384, 32, 5),
                                    (377, 13, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [3, 300])
def test_experts_a_lane(E, G, Gk, score, T):
    """Numbers of experts whose lanes hold 3, 5, 6 or 12, with groups of whole lanes and of others."""
    l, b = data(T, E, E + G, dead=E // 16)
    l[1] = l[1, 0]                                            # equal logits
    l[2, ::2] = l[2, 1]
    rule = dict(score=score, n_group=G, topk_group=Gk, renorm=int(G % 2))
    k = min(6, E // G * Gk)
    check(device(), l, k, rule)
    check(device(), l, k, rule, b)


@pytest.mark.parametrize("T,E,k", [(4864, 8, 2), (4865, 8, 2),       # 32 tokens an SM of 152, 33
                                   (19456, 4, 2), (19457, 4, 2),     # 128, 129
                                   (33, 256, 8), (33, 257, 8), (40, 1024, 8), (1500, 300, 2), (5000, 260, 2)])
@pytest.mark.parametrize("G", [1, 4])
def test_blocks_of_chunks_and_of_eight_tokens(T, E, k, G):
    G = G if E % G == 0 else 1
    l, b = data(T, E, T % 89)
    check(device(), l, k, dict(score="sigmoid", n_group=G, topk_group=max(1, G - 1)), b)
