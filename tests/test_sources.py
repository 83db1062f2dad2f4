"""What the kernels' sources keep to."""
import os

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "serving_router_top_dedupe_gb300", "csrc")


def test_every_cta_loads_its_own_tiles():
    """No copy, commit or arrive goes to other CTAs of a cluster: the library is also loaded where a process drives one of
    several GPUs, and a caller's pages may be any device memory."""
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        assert ".multicast" not in text and "__cluster_dims__" not in text and "mapa." not in text, name
