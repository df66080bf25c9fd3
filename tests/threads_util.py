"""Calls of several threads at once, whose exceptions are the test's own."""
from concurrent.futures import ThreadPoolExecutor


def at_once(calls):
    """Runs the functions, each in a thread of its own, and returns what they return in their order.
    What one of them raises is raised here, when all have ended."""
    with ThreadPoolExecutor(len(calls)) as pool:
        futures = [pool.submit(f) for f in calls]
    return [f.result() for f in futures]
