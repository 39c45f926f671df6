"""Plans of the operators over key/value caches, on stand-in GPUs."""

from flow_matching_action_dm0_b200 import _lib as L
from tests.fake_gpu import gpus, host_library_path  # noqa: F401


def workspace(h, b, tq, tk, hq, hkv, d):
    q = L.rtv_queries(None, None, None, L.RTV_BF16, b, tq, hq, d, tq * hq * d, hq * d, d, tq * hq * d, hq * d, d,
                      d ** -0.5)
    kv = L.rtv_kv(None, None, None, None, L.RTV_BF16, b, tk, hkv, d, tk * hkv * d, hkv * d, d)
    return L.rtv_cross_attention_workspace(h, q, kv)


SHAPES = [(b, tq, tk, 8, 1, d) for d in (64, 128, 256) for b in (1, 2, 3) for tq in (17, 40) for tk in (260, 1000, 4000)]


def test_a_gpus_plans_do_not_depend_on_handles_of_other_gpus(gpus):  # noqa: F811
    """GPU 1 runs no clusters: a handle on it leaves GPU 0's splits, and so its workspaces, as they are."""
    for size in range(2, 17):
        gpus.fake_clusters(1, size, 0)
    first = L.rtv_ops_create(0)
    want = [workspace(first, *s) for s in SHAPES]
    other = L.rtv_ops_create(1)
    there = [workspace(other, *s) for s in SHAPES]
    assert there != want                       # (the shapes' splits do go by it)
    assert [workspace(first, *s) for s in SHAPES] == want
    again = L.rtv_ops_create(0)
    assert [workspace(again, *s) for s in SHAPES] == want
    assert [workspace(other, *s) for s in SHAPES] == there
    for h in (first, other, again):
        L.rtv_ops_destroy(h)
