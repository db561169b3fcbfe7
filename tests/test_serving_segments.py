"""Where long prompts among others are cut, by the room that the scan asks for (no GPU needed)."""
import pytest

import linear_attention_serving_chunk_gb300 as kda


@pytest.fixture(scope="module", autouse=True)
def built():
    kda.build()


@pytest.mark.parametrize("n,total,H,P,cut", [
    # an SM's share of the chunks x column blocks; half of it where it is 48 chunks or more and the
    # whole sequences are two waves of 152 at most
    (6, 32768, 32, 64, 27), (6, 32768, 64, 64, 27), (6, 32768, 96, 64, 40), (6, 32768, 128, 64, 108),
    (12, 65536, 64, 64, 108), (10, 20500, 64, 64, 34), (6, 32768, 32, 128, 27), (6, 32768, 64, 128, 108)])
def test_segments_by_the_share_of_an_sm(n, total, H, P, cut):
    parts = total // (128 * cut)
    assert kda.ssm_workspace_bytes(n, total, H, P, 1, 128) == parts * H * (128 * P + 4) * 4
