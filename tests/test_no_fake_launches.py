"""The refusal tests, whose addresses are fake, do not run where a device could
launch their accepted calls (told here that there is one: collected in a process of
its own, with an availability that says so)."""
import os
import subprocess
import sys

import conftest

RUN = """
import sys, torch, pytest
torch.cuda.is_available = lambda: True
sys.exit(pytest.main(["-q", "-rs", "-p", "no:cacheprovider", *sys.argv[1:]]))
"""


def test_fake_addresses_need_a_machine_without_a_gpu():
    files = [os.path.join(conftest.HERE, f) for f in conftest.NO_DEVICE]
    out = subprocess.run([sys.executable, "-c", RUN, "-k", "refusals or validation or aliasing or temperatures", *files], cwd=conftest.ROOT, capture_output=True, text=True,
                         timeout=600)
    last = out.stdout.strip().splitlines()[-1]
    assert out.returncode == 0 and "skipped" in last and "passed" not in last and "failed" not in last, out.stdout


def test_every_call_that_expects_no_device_is_among_them():
    # an accepted status of "DEVICE" is what marks such a call
    mark = "(OK, " + "DEVICE)"
    for name in os.listdir(conftest.HERE):
        if name.endswith(".py"):
            with open(os.path.join(conftest.HERE, name)) as f:
                assert mark not in f.read() or name in conftest.NO_DEVICE, name
