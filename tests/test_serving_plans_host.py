"""What the decode plans of the serving operators take, seen from the host: the
workspace sizes."""

import compressed_space_attention_b200 as isoq


def test_one_launch_only_where_its_clusters_are_resident():
    """A cluster launch needs no workspace and is taken where the SMs hold all
    its CTAs at once: 148 x 1 at d = 512 with 4 bits, where 32 rows x 4 KV
    heads leave room for one split of a row's 1,024 tokens and two are needed."""
    w = isoq.isoq_decode_window_workspace_size
    assert w(32, 4, 4, 1024, 512, 1024, 0) > 0
    assert w(16, 4, 4, 1024, 512, 1024, 0) == 0      # 64 clusters of two
    assert w(32, 4, 4, 1024, 128, 1024, 0) == 0      # 4 per SM
