"""Host-only: where a paged decode step puts its entry follows the entry0 of the moment."""
import torch

from compressed_sparse_long_csa_b200 import steps


def test_the_place_of_a_fresh_entry_follows_entry0():
    B = 5
    T = {"cache": torch.zeros(B, 50, 16), "entry0": torch.zeros(B, dtype=torch.int32),
         "h_cache": torch.zeros(B, 20, 16), "h_entry0": torch.zeros(B, dtype=torch.int32)}
    D = {"k": 8, "W": 4, "H": 2, "dv": 16}
    steps.page_caches(T, D, "hybrid_pair", page_size=8)
    buffers = {k: T[k].data_ptr() for k in T if "fresh" in k}
    for entries in ([0, 1, 2, 49, 0], [1, 2, 3, 50, -1], [7, 8, 0, 3, -9]):
        for p in ("", "h_"):
            T[p + "entry0"].copy_(torch.tensor(entries, dtype=torch.int32))
            steps._place_fresh(T, p, None)
        for b, e in enumerate(entries):
            if e < 0:
                assert int(T["fresh0"][b]) < 0 and int(T["h_fresh0"][b]) < 0      # the pooling refuses it
                assert T["fresh_entry"][b].tolist() == [-1, -1]
            else:
                assert int(T["fresh0"][b]) == min(e, 1) and int(T["h_fresh0"][b]) == 0
                assert T["fresh_entry"][b].tolist() == ([0, -1] if e == 0 else [-1, e])
    assert buffers == {k: T[k].data_ptr() for k in T if "fresh" in k}             # a captured step keeps them
