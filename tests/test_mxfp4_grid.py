"""Calls of the microscaled 4-bit path whose tiles would be more than a grid has (fewer than 2^32
threads along x) go to the few-row kernel, whose workgroups take turns (CPU only)."""
import pytest

from test_mxfp4_host import ask  # noqa: F401


def grouped(n, d, n_seg, rows, most, glu=0):
    return f"grouped {n} {d} {n_seg} {rows} {most} {glu}"


@pytest.mark.parametrize("line", [grouped(32768, 32, 65535, 65535, 65), grouped(32768, 32, 65535, 65535, 65, 1),
                                  grouped((1 << 27) - 64, 32, 20, 200, 200), grouped(1 << 26, 32, 60, 3000, 3000, 1),
                                  grouped((1 << 27) - 64, 32, 4, 8000, 8000), f"dense {1 << 24} {1 << 16} 32"])
def test_more_tiles_than_a_grid(ask, line):  # noqa: F811
    assert ask([line])[0].startswith("rows")


def test_as_many_as_a_grid(ask):  # noqa: F811
    # 256 columns of tiles, 65533 and 65536 of rows, 256 threads each
    assert ask([grouped(32768, 32, 64510, 65535, 65), grouped(32768, 32, 64513, 65535, 65)]) == ["tile 64", "rows 1 2"]
    # 2^23 - 8192 and 2^23 tiles of 512 threads
    assert ask([grouped(256 * 8192, 32, 4, 261115, 261115), grouped(256 * 8192, 32, 4, 261120, 261120)]) == ["tile 256", "rows 2 2"]
    # 65536 rows of tiles, 127 and 128 columns, 512 threads each
    got = ask([f"dense {1 << 24} 32512 32", f"dense {1 << 24} 32768 32"])
    assert got[0] == "tile 256" and got[1].startswith("rows")
